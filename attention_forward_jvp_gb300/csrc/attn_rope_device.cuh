// Device functions that the rotation (attn_rope.cu) and the cache in 4 bits
// (attn_paged_cache4.cu) share: 16-bit values, the angle of a pair, the
// sequence of a packed token.
#pragma once
#include "attn_paged_kernels.h"
#include "ptx.cuh"

namespace attn {

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (F16) {
    __half2 h;
    *reinterpret_cast<uint32_t*>(&h) = w;
    return __half22float2(h);
  } else {
    return make_float2(bf16_lo(w), bf16_hi(w));
  }
}

template <bool F16>
__device__ __forceinline__ float widen(uint16_t h) {
  if constexpr (F16) return __half2float(__ushort_as_half(h));
  else return __uint_as_float(static_cast<uint32_t>(h) << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t narrow(float f) {
  if constexpr (F16) return __half_as_ushort(__float2half_rn(f));
  else return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// cos and sin (times the output scale) of pair `pair` at position pos
__device__ __forceinline__ float2 turn(const RopeSpec& r, int pair, int pos) {
  const unsigned long long ph =
      r.steps[pair] * static_cast<unsigned long long>(static_cast<long long>(pos));
  float s, c;
  __sincosf(static_cast<float>(static_cast<int>(ph >> 32)) * 1.462918079267160e-9f, &s, &c);  // pi 2^-31
  if (r.inverse) s = -s;
  return make_float2(c * r.scale, s * r.scale);
}

// The same to the last bits, for a rounding to 4 bits, which has steps that
// __sincosf's error takes one more time in 10^5 to the wrong side of: the nearest
// quarter of a turn in whole numbers, and CUDA's sincospif of what is left.
__device__ __forceinline__ float2 turn_close(const RopeSpec& r, int pair, int pos) {
  const unsigned long long ph =
      r.steps[pair] * static_cast<unsigned long long>(static_cast<long long>(pos));
  const uint32_t at = static_cast<uint32_t>(ph >> 32), quarter = (at + 0x20000000u) >> 30;
  float s, c;
  sincospif(static_cast<float>(static_cast<int>(at - (quarter << 30))) * 4.656612873077393e-10f, &s, &c);  // 2^-31
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  c = (quarter + 1) & 2 ? -x : x;
  s = quarter & 2 ? -y : y;
  if (r.inverse) s = -s;
  return make_float2(c * r.scale, s * r.scale);
}

// The sequence of packed token t, the last b < n_seq with offsets[b] <= t,
// for a whole warp: 32 offsets at a time for the first lane's token, then
// step by step for the others', which lie behind it (or have no part in the
// answer and lie before).  All lanes take part.
__device__ __forceinline__ int sequence_of(const int* offsets, int n_seq, long long t) {
  const int lane = threadIdx.x & 31;
  const long long t0 = __shfl_sync(0xffffffffu, t, 0);
  int b = 0, n = n_seq;  // the one sought is in [b, b + n)
  while (n > 1) {
    const int k = (n + 31) / 32;
    const bool below = lane * k < n && offsets[b + lane * k] <= t0;
    const int c = max(__popc(__ballot_sync(0xffffffffu, below)) - 1, 0);
    b += c * k;
    n = min(k, n - c * k);
  }
  while (b + 1 < n_seq && offsets[b + 1] <= t) ++b;
  return b;
}

}  // namespace attn
