// The append to a cache in 4 bits (attn_paged_append4), and a cache of either
// kind read back as dense tensors (attn_paged_gather, attn_paged_gather4).
//
// Append: of a group of 64 neighbouring elements (32 where D = 32), after the
// rotation, m = fp16(min), s = fp16((max - m) / 15), n = round((x - m) / s) in
// 0 .. 15, with the quotients of IEEE's division, so that n is a function of x
// alone: x - m times 1 / s rounds to the same n unless it lies within 10^-4 of
// a half (it is off by 4 10^-6 at most), and is divided where it does.  Eight
// elements to a thread, the row of a head to D / 8 neighbouring lanes of one
// warp: the group's extremes come from three exchanges between lanes, and the
// element that x turns with from another lane of the row.  A warp takes heads
// of one token, whose angles it computes once, the rows of several on their way.
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
constexpr int kWarps = 8, kAppendUnroll = 4;

// eight neighbouring elements: VEC says that they are one 16-byte word
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* x, bool live) {
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (!live) return w;
  if constexpr (VEC) return *reinterpret_cast<const uint4*>(x);
  uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = x[2 * i] | static_cast<uint32_t>(x[2 * i + 1]) << 16;
  return w;
}
template <bool F16>
__device__ __forceinline__ void widen8(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2<F16>(u[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
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
  // f: the elements w; x: the row in memory.  All lanes take part.
  template <bool F16, bool VEC>
  __device__ __forceinline__ void apply(const RopeSpec& r, int d0, const uint16_t* x, bool live, const uint4& w,
                                        float (&f)[8]) const {
    widen8<F16>(w, f);
    if (r.rot == 0) return;
    float o[8];
    if constexpr (VEC) {  // rot a multiple of 16: a lane's elements turn with another lane's, or with one another
      if (r.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = f[j ^ 1];
      } else {
        const int shift = d0 < r.rot / 2 ? r.rot / 16 : (d0 < r.rot ? -(r.rot / 16) : 0);
        const int from = (threadIdx.x & 31) + shift;
        widen8<F16>(make_uint4(__shfl_sync(kAll, w.x, from), __shfl_sync(kAll, w.y, from), __shfl_sync(kAll, w.z, from),
                               __shfl_sync(kAll, w.w, from)),
                    o);
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
    const float inv = __frcp_rn(sf);  // (finite: s is 2^-24 or more)
    bool near = false;
    float n[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = (f[j] - mf) * inv;
      n[j] = rintf(y);
      near = near || fabsf(y - n[j]) > 0.4999f;
    }
    if (near) {
#pragma unroll
      for (int j = 0; j < 8; ++j) n[j] = rintf(__fdiv_rn(f[j] - mf, sf));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)  // (2^23 + n: n in the low bits)
      word |= (__float_as_uint(fminf(fmaxf(n[j], 0.f), 15.f) + 8388608.f) & 15u) << (4 * j);
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

  // heads of q, of k and of v, one after the other: `use` for each row that
  // this lane has eight elements of, those of U rows on their way
  constexpr int U = VEC ? kAppendUnroll : 1;
  const int first = blockIdx.y * p.heads_per_split;
  const int last = min(first + p.heads_per_split, p.Hq + 2 * p.Hkv);
  auto heads = [&](const uint16_t* base, long long stride, int D, int lo, int hi, auto use) {
    const int L = D / 8, R = 32 / L, d0 = 8 * (lane & (L - 1)), r = lane / L;
#pragma unroll 1
    for (int h0 = lo; h0 < hi; h0 += R * U) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * R + r;
        w[u] = load8<VEC>(base + (h < hi ? h : lo) * stride + d0, h < hi);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * R + r;
        if (h0 + u * R < hi) use(w[u], base + (h < hi ? h : lo) * stride, h, h < hi, d0);
      }
    }
  };
  Turn8 turned;
  if (first < p.Hq + p.Hkv && pos >= 0) turned.angles(p.r, 8 * (lane & (p.Dqk / 8 - 1)), static_cast<int>(pos));
  if (pos >= 0) {
    heads(p.q + t * p.qs[0], p.qs[1], p.Dqk, first, min(last, p.Hq),
          [&](const uint4& w, const uint16_t* x, int h, bool live, int d0) {
            float f[8];
            turned.apply<F16, VEC>(p.r, d0, x, live, w, f);
            __syncwarp();  // in place: the row has been read
            if (live) store8<F16, VEC>(p.q_out + t * p.qos[0] + h * p.qos[1] + d0, f);
          });
  } else {  // no position: zeros
    const float zero[8] = {};
    const int L = p.Dqk / 8;
    for (int h = first + lane / L; h < min(last, p.Hq); h += 32 / L)
      store8<F16, VEC>(p.q_out + t * p.qos[0] + h * p.qos[1] + 8 * (lane & (L - 1)), zero);
  }
  if (!placed) return;
  heads(p.k + t * p.ks[0], p.ks[1], p.Dqk, max(first - p.Hq, 0), min(last - p.Hq, p.Hkv),
        [&](const uint4& w, const uint16_t* x, int h, bool live, int d0) {
          float f[8];
          turned.apply<F16, VEC>(p.r, d0, x, live, w, f);
          store_row4(p4.k, page, h, slot, p.Dqk, d0, live, f);
        });
  heads(p.v + t * p.vs[0], p.vs[1], p.Dv, max(first - p.Hq - p.Hkv, 0), min(last - p.Hq - p.Hkv, p.Hkv),
        [&](const uint4& w, const uint16_t*, int h, bool live, int d0) {
          float f[8];
          widen8<F16>(w, f);
          store_row4(p4.v, page, h, slot, p.Dv, d0, live, f);
        });
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
    // n in the low bits of a half is the subnormal n 2^-24, 16 n that of an odd
    // element; n s is exact (15 bits)
    const float m1 = __half2float(__ushort_as_half(m)), s1 = __half2float(__ushort_as_half(s)) * 16777216.f;
    const float s16 = s1 * 0.0625f;
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // elements 2 i, 2 i + 1 and 4 further on
      const uint32_t a = w >> (8 * i) & 0x000f000fu, b = w >> (8 * i) & 0x00f000f0u;
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
      u[i] = pack2<F16>(fmaf(x.x, s1, m1), fmaf(y.x, s16, m1));
      u[2 + i] = pack2<F16>(fmaf(x.y, s1, m1), fmaf(y.y, s16, m1));
    }
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
