// The append to a cache in 4 bits (attn_paged_append4), and a cache of either
// kind read back as dense tensors (attn_paged_gather, attn_paged_gather4).
//
// Append: of a group of 64 neighbouring elements (32 where D = 32), after the
// rotation, m = fp16(min), s = fp16((max - m) / 15), n = round((x - m) / s) in
// 0 .. 15; the divisions are IEEE's, so that n is a function of x alone.  Eight
// elements to a thread, the row of a head to D / 8 neighbouring lanes of one
// warp: the group's extremes come from three exchanges between lanes, and the
// element that x turns with from another lane of the row.  A warp takes heads
// of one token, whose angles it computes once.
//
// Gather: a thread owns eight elements of one token and walks over the heads,
// several loads in flight.
//
// Both are bound by memory: a new token's row is read in 16 bits and written in
// 4.5, the gather's read in 4.5 or 16 and written in 16.
#include <type_traits>

#include "attn_paged_cache_kernels.h"
#include "attn_rope_device.cuh"
#include "ptx.cuh"

namespace attn {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;

// eight neighbouring elements, of which VEC says that they are one 16-byte word
template <bool F16, bool VEC>
__device__ __forceinline__ void load8(const uint16_t* x, bool live, float (&f)[8]) {
  if constexpr (VEC) {
    const uint4 w = live ? *reinterpret_cast<const uint4*>(x) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2<F16>(u[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = live ? widen<F16>(x[i]) : 0.f;
  }
}
template <bool F16, bool VEC>
__device__ __forceinline__ void store8(uint16_t* y, const float (&f)[8]) {
  if constexpr (VEC) {
    *reinterpret_cast<uint4*>(y) = make_uint4(pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]),
                                              pack2<F16>(f[6], f[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = narrow<F16>(f[i]);
  }
}

// The rotation of a row of which this lane holds elements d0 .. d0 + 7
struct Turn8 {
  float2 cs[8];

  __device__ __forceinline__ void angles(const RopeSpec& r, int d0, int pos) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = d0 + j;
      if (d < r.rot) {
        const int pair = r.interleaved ? d >> 1 : (d < r.rot / 2 ? d : d - r.rot / 2);
        cs[j] = turn(r, pair, pos);
        const bool first = r.interleaved ? !(d & 1) : d < r.rot / 2;
        if (first) cs[j].y = -cs[j].y;  // x cos - other sin; the second of a pair x cos + other sin
      } else {
        cs[j] = make_float2(1.f, 0.f);
      }
    }
  }
  // f: this lane's elements; x: the row in memory.  All lanes take part.
  template <bool F16, bool VEC>
  __device__ __forceinline__ void apply(const RopeSpec& r, int d0, const uint16_t* x, bool live, float (&f)[8]) const {
    float o[8];
    if constexpr (VEC) {  // rot a multiple of 16: a lane's elements turn with another lane's, or with one another
      if (r.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = f[j ^ 1];
      } else {
        const int shift = d0 < r.rot / 2 ? r.rot / 16 : (d0 < r.rot ? -(r.rot / 16) : 0);
        const int from = (threadIdx.x & 31) + shift;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(kAll, f[j], from);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int d = d0 + j;
        o[j] = 0.f;
        if (live && d < r.rot)
          o[j] = widen<F16>(x[r.interleaved ? d ^ 1 : (d < r.rot / 2 ? d + r.rot / 2 : d - r.rot / 2)]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = d0 + j < r.rot ? f[j] * cs[j].x + o[j] * cs[j].y : f[j];
  }
};

// Rounds a row whose elements d0 .. d0 + 7 this lane holds, and stores it.
// All lanes take part; d: elements of the row.
__device__ __forceinline__ void store_row4(const Pool4& pool, long long page, int h, long long slot, int d, int d0,
                                           bool live, float (&f)[8]) {
  const int lane = threadIdx.x & 31;
  const int lanes = d < 64 ? 4 : 8;  // of a group
  constexpr float kMost = 65504.f;
  bool odd = false;
  float lo = 3.402823466e38f, hi = -3.402823466e38f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    odd = odd || !(fabsf(f[j]) <= 3.402823466e38f);
    f[j] = fminf(fmaxf(f[j], -kMost), kMost);
    lo = fminf(lo, f[j]);
    hi = fmaxf(hi, f[j]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float a = __shfl_xor_sync(kAll, lo, o), b = __shfl_xor_sync(kAll, hi, o);
    if (o < lanes) {
      lo = fminf(lo, a);
      hi = fmaxf(hi, b);
    }
  }
  const unsigned odds = __ballot_sync(kAll, odd) >> (lane & ~(lanes - 1)) & ((1u << lanes) - 1);
  if (!live) return;
  __half m = __float2half_rn(lo);
  const float mf = __half2float(m);
  __half s = __float2half_rn(__fdiv_rn(hi - mf, 15.f));
  const float sf = __half2float(s);
  uint32_t word = 0;
  if (odds) {
    m = s = __ushort_as_half(0x7fff);
  } else if (sf > 0.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float n = fminf(fmaxf(rintf(__fdiv_rn(f[j] - mf, sf)), 0.f), 15.f);
      word |= static_cast<uint32_t>(n) << (4 * j);
    }
  }
  uint8_t* codes = pool.codes + page * pool.st[0] + h * pool.st[1] + slot * pool.st[2];
  *reinterpret_cast<uint32_t*>(codes + d0 / 2) = word;
  if ((lane & (lanes - 1)) == 0) {
    uint16_t* to = pool.scales + page * pool.ss[0] + h * pool.ss[1] + slot * pool.ss[2];
    const int g = d0 / 64;
    to[g] = __half_as_ushort(s);
    to[groups4(d) + g] = __half_as_ushort(m);
  }
}

template <bool F16, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) append4_kernel(const __grid_constant__ Append4Params p4) {
  griddep_wait();
  griddep_launch_dependents();
  const AppendParams& p = p4.a;
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  // the token's sequence and position
  long long b = t, pos = 0;
  bool idle = false;
  if (p.offsets != nullptr) {
    if (t >= p.offsets[p.B]) return;
    b = sequence_of(p.offsets, p.B, t);
    pos = p.seq_lens[b] - static_cast<long long>(p.offsets[b + 1]) + t;
  } else {
    pos = static_cast<long long>(p.seq_lens[b]) - 1;
    idle = pos == -1;
  }
  // its place in the pool
  long long page = -1, slot = 0;
  if (pos >= 0 && pos < static_cast<long long>(p.max_pages) * p.page_size) {
    const int e = static_cast<int>(pos / p.page_size);
    slot = pos - static_cast<long long>(e) * p.page_size;
    page = p.page_table[b * p.table_stride + e];
  }
  const bool placed = page >= 0 && page < p.n_pages;
  if (!placed && !idle && lane == 0 && blockIdx.y == 0) *p.err = 1;

  // heads of q, of k and of v, one after the other
  const int first = blockIdx.y * p.heads_per_split;
  const int last = min(first + p.heads_per_split, p.Hq + 2 * p.Hkv);
  {
    const int L = p.Dqk / 8, R = 32 / L, d0 = 8 * (lane & (L - 1)), r = lane / L;
    Turn8 turned;
    if (first < p.Hq + p.Hkv && pos >= 0) turned.angles(p.r, d0, static_cast<int>(pos));
    for (int h = first + r, end = min(last, p.Hq); h - r < end; h += R) {
      const bool live = h < end;
      const uint16_t* x = p.q + t * p.qs[0] + (live ? h : first) * p.qs[1];
      uint16_t* y = p.q_out + t * p.qos[0] + (live ? h : first) * p.qos[1];
      float f[8] = {};
      if (pos >= 0) {
        load8<F16, VEC>(x + d0, live, f);
        turned.apply<F16, VEC>(p.r, d0, x, live, f);
        __syncwarp();  // in place: the row has been read
      }
      if (live) store8<F16, VEC>(y + d0, f);
    }
    if (!placed) return;
    for (int h = max(first - p.Hq, 0) + r, end = min(last - p.Hq, p.Hkv); h - r < end; h += R) {
      const bool live = h < end;
      const uint16_t* x = p.k + t * p.ks[0] + (live ? h : 0) * p.ks[1];
      float f[8];
      load8<F16, VEC>(x + d0, live, f);
      turned.apply<F16, VEC>(p.r, d0, x, live, f);
      store_row4(p4.k, page, h, slot, p.Dqk, d0, live, f);
    }
  }
  {
    const int L = p.Dv / 8, R = 32 / L, d0 = 8 * (lane & (L - 1)), r = lane / L;
    for (int h = max(first - p.Hq - p.Hkv, 0) + r, end = min(last - p.Hq - p.Hkv, p.Hkv); h - r < end; h += R) {
      const bool live = h < end;
      const uint16_t* x = p.v + t * p.vs[0] + (live ? h : 0) * p.vs[1];
      float f[8];
      load8<F16, VEC>(x + d0, live, f);
      store_row4(p4.v, page, h, slot, p.Dv, d0, live, f);
    }
  }
}

// ------------------------------------------------------------------- gather
constexpr int kGatherThreads = 256, kGatherUnroll = 4;

// eight elements of a row in 16 bits
struct Held16 {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* pool, const long long (&st)[3], long long page, int h,
                                       long long slot, int d0) {
    w = *reinterpret_cast<const uint4*>(pool + page * st[0] + h * st[1] + slot * st[2] + d0);
  }
  template <bool F16>
  __device__ __forceinline__ uint4 value() const {
    return w;
  }
};
// eight elements of a row in 4 bits
struct Held4 {
  uint32_t w;
  uint16_t s, m;
  __device__ __forceinline__ void load(const Pool4& pool, long long page, int h, long long slot, int d, int d0) {
    w = *reinterpret_cast<const uint32_t*>(pool.codes + page * pool.st[0] + h * pool.st[1] + slot * pool.st[2] + d0 / 2);
    const uint16_t* at = pool.scales + page * pool.ss[0] + h * pool.ss[1] + slot * pool.ss[2] + d0 / 64;
    s = at[0];
    m = at[groups4(d)];
  }
  template <bool F16>
  __device__ __forceinline__ uint4 value() const {
    const float sf = __half2float(__ushort_as_half(s)), mf = __half2float(__ushort_as_half(m));
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // (n s is exact: 15 bits)
      u[i] = pack2<F16>(fmaf(static_cast<float>(w >> (8 * i) & 15u), sf, mf),
                        fmaf(static_cast<float>(w >> (8 * i + 4) & 15u), sf, mf));
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

template <int BITS, bool F16>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int items = max(p.Dqk, p.Dv) / 8;  // a power of two, at most 32
  const int row_in_block = threadIdx.x / items, d0 = 8 * (threadIdx.x & (items - 1));
  const long long t0 = static_cast<long long>(blockIdx.x) * (kGatherThreads / items);
  long long t = t0 + row_in_block;
  const bool none = t >= p.T;
  if (none) t = t0;  // (takes part in the search)
  const long long b = sequence_of(p.offsets, p.B, t);
  if (none || t >= p.offsets[p.B]) return;
  const long long pos = p.seq_lens[b] - static_cast<long long>(p.offsets[b + 1]) + t;
  long long page = -1, slot = 0;
  if (pos >= 0 && pos < static_cast<long long>(p.max_pages) * p.page_size) {
    const int e = static_cast<int>(pos / p.page_size);
    slot = pos - static_cast<long long>(e) * p.page_size;
    page = p.page_table[b * p.table_stride + e];
  }
  const bool placed = page >= 0 && page < p.n_pages;
  if (!placed && d0 == 0 && blockIdx.y == 0) *p.err = 1;
  const int first = blockIdx.y * p.heads_per_split, last = min(first + p.heads_per_split, p.Hkv);
  const bool in_k = d0 < p.Dqk, in_v = d0 < p.Dv;
  uint16_t* ko = p.k_out + t * p.ko[1] + d0;
  uint16_t* vo = p.v_out + t * p.vo[1] + d0;
  if (!placed) {
    for (int h = first; h < last; ++h) {
      if (in_k) *reinterpret_cast<uint4*>(ko + h * p.ko[0]) = make_uint4(0u, 0u, 0u, 0u);
      if (in_v) *reinterpret_cast<uint4*>(vo + h * p.vo[0]) = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  constexpr int U = kGatherUnroll;
  using Held = typename std::conditional<BITS == 4, Held4, Held16>::type;
#pragma unroll 1
  for (int h0 = first; h0 < last; h0 += U) {
    Held k[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u < last ? h0 + u : h0;
      if constexpr (BITS == 4) {
        if (in_k) k[u].load(p.k, page, h, slot, p.Dqk, d0);
        if (in_v) v[u].load(p.v, page, h, slot, p.Dv, d0);
      } else {
        if (in_k) k[u].load(p.k16, p.kp, page, h, slot, d0);
        if (in_v) v[u].load(p.v16, p.vp, page, h, slot, d0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u;
      if (h >= last) break;
      if (in_k) *reinterpret_cast<uint4*>(ko + h * p.ko[0]) = k[u].template value<F16>();
      if (in_v) *reinterpret_cast<uint4*>(vo + h * p.vo[0]) = v[u].template value<F16>();
    }
  }
}

template <class P>
cudaError_t launch(void (*kernel)(P), const P& p, dim3 grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_append4(const Append4Params& p, bool vec, bool f16, int splits, cudaStream_t stream) {
  const long long blocks = (p.a.T + kWarps - 1) / kWarps;
  const dim3 grid(static_cast<unsigned>(blocks), splits);
  if (f16) return launch(vec ? append4_kernel<true, true> : append4_kernel<true, false>, p, grid, kWarps * 32, stream);
  return launch(vec ? append4_kernel<false, true> : append4_kernel<false, false>, p, grid, kWarps * 32, stream);
}

cudaError_t launch_gather(const GatherParams& p, int bits, bool f16, int splits, cudaStream_t stream) {
  const int rows = kGatherThreads / ((p.Dqk > p.Dv ? p.Dqk : p.Dv) / 8);
  const dim3 grid(static_cast<unsigned>((p.T + rows - 1) / rows), splits);
  if (bits == 16) return launch(gather_kernel<16, false>, p, grid, kGatherThreads, stream);
  return launch(f16 ? gather_kernel<4, true> : gather_kernel<4, false>, p, grid, kGatherThreads, stream);
}

}  // namespace attn
