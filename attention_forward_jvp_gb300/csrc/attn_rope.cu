// Rotary positions (attn_rope) and the append to the paged cache
// (attn_paged_append).
//
// Pair i of a token at position p turns by the angle p * w_i.  The kernels
// hold w_i as a 64-bit fraction of a full turn, so that p * step modulo 2^64
// is the angle modulo a full turn exactly, at any position, in three integer
// multiplications; its upper 32 bits, taken as a signed fraction of half a
// turn and multiplied by pi, go to __sincosf.  (p * w_i in fp32 is off by
// 2^-24 p: 0.008 rad at position 131072.)  The fraction and the product are
// rounded to fp32, 3 10^-7 together, and __sincosf is within 2^-21.1 on
// [-pi, pi]: 8 10^-7, against the 2^-12 relative of the finer of the two
// storage types.  (sincospif, exact to 10^-7 but five times the
// instructions, cost 1 to 4 % at the sizes below.)
//
// Both are bound by memory: an element is read once and written once.  A
// thread owns two 16-byte pieces of one token, half a row (of the rotated
// part, or of the rest) apart: the pieces that turn together where pairs are
// half-split, and neighbouring threads on neighbouring pieces in any case.
// It computes its eight angles once, behind the first loads, and walks over
// the heads with them in registers, two heads of 16-byte loads in flight and
// four blocks on an SM (four heads and two blocks were slower: 47 us for 45);
// a table of cos and sin, the alternative, is a second stream to read and has
// to end at some position.
#include "attn_paged_kernels.h"
#include "attn_rope_device.cuh"
#include "ptx.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256, kBlocks = 4;

struct Piece {
  uint4 a, b;
};
__device__ __forceinline__ Piece load_piece(const uint16_t* x, int d1) {
  return {*reinterpret_cast<const uint4*>(x), *reinterpret_cast<const uint4*>(x + d1)};
}
__device__ __forceinline__ void store_piece(uint16_t* y, int d1, const Piece& v) {
  *reinterpret_cast<uint4*>(y) = v.a;
  *reinterpret_cast<uint4*>(y + d1) = v.b;
}

// Eight pairs.  Half-split: element j of a with element j of b;
// interleaved: the four pairs of neighbours of a, then those of b.
template <bool F16, bool INTER>
__device__ __forceinline__ void rotate_piece(Piece& v, const float2 (&cs)[8]) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&v.a);
  uint32_t* b = reinterpret_cast<uint32_t*>(&v.b);
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? a[i] : b[i - 4];
      const float2 x = unpack2<F16>(w);
      w = pack2<F16>(x.x * cs[i].x - x.y * cs[i].y, x.x * cs[i].y + x.y * cs[i].x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2<F16>(a[i]), y = unpack2<F16>(b[i]);
      const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
      a[i] = pack2<F16>(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
      b[i] = pack2<F16>(x.x * c0.y + y.x * c0.x, x.y * c1.y + y.y * c1.x);
    }
  }
}

// The angles of a thread's piece, computed when first needed: behind loads
struct Angles {
  float2 cs[8];
  bool have = false;
  // of item `item` of the rotated part
  template <bool INTER>
  __device__ __forceinline__ void need(const RopeSpec& r, int item, int pos) {
    if (have) return;
    have = true;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      cs[i] = turn(r, INTER ? 4 * item + (i & 3) + (i < 4 ? 0 : r.rot / 4) : 8 * item + i, pos);
  }
};

// n heads of one piece: rotated, or copied
template <bool F16, bool INTER>
__device__ __forceinline__ void walk_heads(const uint16_t* x, long long xh, uint16_t* y, long long yh, int n, int d1,
                                           bool turned, Angles& a, const RopeSpec& r, int item, int pos) {
  constexpr int U = kRopeUnroll;
  int h = 0;
#pragma unroll 1
  for (; h + U <= n; h += U) {
    Piece v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = load_piece(x + u * xh, d1);
    if (turned) {
      a.template need<INTER>(r, item, pos);
#pragma unroll
      for (int u = 0; u < U; ++u) rotate_piece<F16, INTER>(v[u], a.cs);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) store_piece(y + u * yh, d1, v[u]);
    x += U * xh;
    y += U * yh;
  }
#pragma unroll 1
  for (; h < n; ++h, x += xh, y += yh) {
    Piece v = load_piece(x, d1);
    if (turned) {
      a.template need<INTER>(r, item, pos);
      rotate_piece<F16, INTER>(v, a.cs);
    }
    store_piece(y, d1, v);
  }
}

// The same, element by element: a pair (d0, d1) turned, or element d0 copied
template <bool F16>
__device__ __forceinline__ void walk_heads_scalar(const uint16_t* x, long long xh, uint16_t* y, long long yh, int n,
                                                  int d0, int d1, bool turned, float2 cs) {
  for (int h = 0; h < n; ++h, x += xh, y += yh) {
    if (turned) {
      const float a = widen<F16>(x[d0]), b = widen<F16>(x[d1]);
      y[d0] = narrow<F16>(a * cs.x - b * cs.y);
      y[d1] = narrow<F16>(a * cs.y + b * cs.x);
    } else {
      y[d0] = x[d0];
    }
  }
}

// pieces (VEC) or pairs and single elements (scalar) of a row of d elements
template <bool VEC>
__device__ __forceinline__ int items_of(int d, int rot) {
  return VEC ? d / 16 : d - rot / 2;
}

template <bool F16, bool INTER, bool VEC>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_kernel(const __grid_constant__ RopeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int items = items_of<VEC>(p.D, p.r.rot);
  // a block holds whole rows, or pieces of one when a row has more items
  // than it has threads
  const int per_row = items < kThreads ? items : kThreads;
  const int row_in_block = threadIdx.x / per_row;
  long long row = static_cast<long long>(blockIdx.x) * (kThreads / per_row) + row_in_block;
  const bool idle = row_in_block >= kThreads / per_row || row >= p.rows;
  if (idle) row = static_cast<long long>(blockIdx.x) * (kThreads / per_row);  // (takes part in the search)
  const long long b = p.N == p.rows ? 0 : row / p.N;
  const long long n = row - b * p.N;
  int pos = static_cast<int>(n);
  if (p.offsets != nullptr) {
    const int seq = sequence_of(p.offsets, p.n_seq, n);
    if (n >= p.offsets[p.n_seq]) return;
    pos -= p.offsets[seq];
  }
  if (idle) return;
  if (p.positions != nullptr) pos = p.positions[b * p.ps[0] + n * p.ps[1]];

  for (int item = threadIdx.x - row_in_block * per_row; item < items; item += per_row) {
    Angles angles;
    bool turned;
    int d0, d1;
    if constexpr (VEC) {
      turned = item < p.r.rot / 16;
      d0 = turned ? 8 * item : p.r.rot / 2 + 8 * item;  // behind rot: 8 (item - rot / 16) further
      d1 = (turned ? p.r.rot : p.D - p.r.rot) / 2;
    } else {
      turned = item < p.r.rot / 2;
      d0 = turned ? (INTER ? 2 * item : item) : item + p.r.rot / 2;
      d1 = INTER ? d0 + 1 : d0 + p.r.rot / 2;
      if (turned) angles.cs[0] = turn(p.r, item, pos);
    }
    const int first = blockIdx.y * p.heads_per_split;
    const int last = min(first + p.heads_per_split, p.heads);
    int h0 = 0;
#pragma unroll 1
    for (int t = 0; t < p.n_tensors; ++t) {
      const RopeTensor& a = p.t[t];
      const int lo = max(first - h0, 0), hi = min(last - h0, a.H);
      h0 += a.H;
      if (lo >= hi) continue;
      const uint16_t* x = a.x + b * a.xs[0] + lo * a.xs[1] + n * a.xs[2];
      uint16_t* y = a.y + b * a.ys[0] + lo * a.ys[1] + n * a.ys[2];
      if (!turned && x == y) continue;  // in place: nothing to copy
      if constexpr (VEC)
        walk_heads<F16, INTER>(x + d0, a.xs[1], y + d0, a.ys[1], hi - lo, d1, turned, angles, p.r, item, pos);
      else
        walk_heads_scalar<F16>(x, a.xs[1], y, a.ys[1], hi - lo, d0, d1, turned, angles.cs[0]);
    }
  }
}

template <bool F16, bool INTER, bool VEC>
__global__ void __launch_bounds__(kThreads, kBlocks) append_kernel(const __grid_constant__ AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int items_qk = items_of<VEC>(p.Dqk, p.r.rot), items_v = items_of<VEC>(p.Dv, 0);
  const int items = max(items_qk, items_v);
  const int per_row = items < kThreads ? items : kThreads;
  const int row_in_block = threadIdx.x / per_row;
  long long t = static_cast<long long>(blockIdx.x) * (kThreads / per_row) + row_in_block;
  const bool none = row_in_block >= kThreads / per_row || t >= p.T;
  if (none) t = static_cast<long long>(blockIdx.x) * (kThreads / per_row);  // (takes part in the search)
  const int item = threadIdx.x - row_in_block * per_row;  // items <= 256: every one has its thread

  // the token's sequence and position
  long long b = t, pos = 0;
  bool idle = false;
  if (p.offsets != nullptr) {
    b = sequence_of(p.offsets, p.B, t);
    if (t >= p.offsets[p.B]) return;
    pos = p.seq_lens[b] - static_cast<long long>(p.offsets[b + 1]) + t;
  } else {
    pos = static_cast<long long>(p.seq_lens[b]) - 1;
    idle = pos == -1;
  }
  if (none) return;
  // its place in the pool
  long long page = -1, slot = 0;
  if (pos >= 0 && pos < static_cast<long long>(p.max_pages) * p.page_size) {
    const int e = static_cast<int>(pos / p.page_size);
    slot = pos - static_cast<long long>(e) * p.page_size;
    page = p.page_table[b * p.table_stride + e];
  }
  const bool placed = page >= 0 && page < p.n_pages;
  if (!placed && !idle && item == 0 && blockIdx.y == 0) *p.err = 1;

  Angles angles;
  const bool turned = item < (VEC ? p.r.rot / 16 : p.r.rot / 2);
  int d0, d1;
  if constexpr (VEC) {
    d0 = turned ? 8 * item : p.r.rot / 2 + 8 * item;
    d1 = (turned ? p.r.rot : p.Dqk - p.r.rot) / 2;
  } else {
    d0 = turned ? (INTER ? 2 * item : item) : item + p.r.rot / 2;
    d1 = INTER ? d0 + 1 : d0 + p.r.rot / 2;
    if (turned && pos >= 0) angles.cs[0] = turn(p.r, item, static_cast<int>(pos));
  }

  // heads of q, of k and of v, one after the other
  const int first = blockIdx.y * p.heads_per_split;
  const int last = min(first + p.heads_per_split, p.Hq + 2 * p.Hkv);
  {
    const int lo = first, hi = min(last, p.Hq);
    if (lo < hi && item < items_qk) {
      const uint16_t* x = p.q + t * p.qs[0] + lo * p.qs[1];
      uint16_t* y = p.q_out + t * p.qos[0] + lo * p.qos[1];
      if (pos < 0) {  // no position: zeros
        for (int h = lo; h < hi; ++h, y += p.qos[1]) {
          if constexpr (VEC) {
            store_piece(y + d0, d1, Piece{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)});
          } else {
            y[d0] = 0;
            if (turned) y[d1] = 0;
          }
        }
      } else if (turned || x != y) {
        if constexpr (VEC)
          walk_heads<F16, INTER>(x + d0, p.qs[1], y + d0, p.qos[1], hi - lo, d1, turned, angles, p.r, item, static_cast<int>(pos));
        else
          walk_heads_scalar<F16>(x, p.qs[1], y, p.qos[1], hi - lo, d0, d1, turned, angles.cs[0]);
      }
    }
  }
  if (!placed) return;
  {
    const int lo = max(first - p.Hq, 0), hi = min(last - p.Hq, p.Hkv);
    if (lo < hi && item < items_qk) {
      const uint16_t* x = p.k + t * p.ks[0] + lo * p.ks[1];
      uint16_t* y = p.k_pool + page * p.kp[0] + lo * p.kp[1] + slot * p.kp[2];
      if constexpr (VEC)
        walk_heads<F16, INTER>(x + d0, p.ks[1], y + d0, p.kp[1], hi - lo, d1, turned, angles, p.r, item, static_cast<int>(pos));
      else
        walk_heads_scalar<F16>(x, p.ks[1], y, p.kp[1], hi - lo, d0, d1, turned, angles.cs[0]);
    }
  }
  {
    const int lo = max(first - p.Hq - p.Hkv, 0), hi = min(last - p.Hq - p.Hkv, p.Hkv);
    if (lo < hi && item < items_v) {
      const uint16_t* x = p.v + t * p.vs[0] + lo * p.vs[1];
      uint16_t* y = p.v_pool + page * p.vp[0] + lo * p.vp[1] + slot * p.vp[2];
      if constexpr (VEC)
        walk_heads<F16, INTER>(x + 8 * item, p.vs[1], y + 8 * item, p.vp[1], hi - lo, p.Dv / 2, false, angles, p.r, 0, 0);
      else
        walk_heads_scalar<F16>(x, p.vs[1], y, p.vp[1], hi - lo, item, item, false, angles.cs[0]);
    }
  }
}

template <class P>
cudaError_t launch(void (*kernel)(P), const P& p, dim3 grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class P, template <bool, bool, bool> class K>
cudaError_t pick(const P& p, bool vec, bool f16, dim3 grid, cudaStream_t stream) {
  const bool in = p.r.interleaved != 0;
  if (f16) {
    if (in) return launch(vec ? K<true, true, true>::fn : K<true, true, false>::fn, p, grid, stream);
    return launch(vec ? K<true, false, true>::fn : K<true, false, false>::fn, p, grid, stream);
  }
  if (in) return launch(vec ? K<false, true, true>::fn : K<false, true, false>::fn, p, grid, stream);
  return launch(vec ? K<false, false, true>::fn : K<false, false, false>::fn, p, grid, stream);
}
template <bool F16, bool INTER, bool VEC>
struct RopeK {
  static constexpr auto fn = rope_kernel<F16, INTER, VEC>;
};
template <bool F16, bool INTER, bool VEC>
struct AppendK {
  static constexpr auto fn = append_kernel<F16, INTER, VEC>;
};

// blocks over the rows
long long row_blocks(long long rows, int items) {
  const int per_row = items < kThreads ? items : kThreads;
  const int rows_per_block = kThreads / per_row;
  return (rows + rows_per_block - 1) / rows_per_block;
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool vec, bool f16, int splits, cudaStream_t stream) {
  const long long blocks = row_blocks(p.rows, vec ? p.D / 16 : p.D - p.r.rot / 2);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return pick<RopeParams, RopeK>(p, vec, f16, dim3(static_cast<unsigned>(blocks), splits), stream);
}

cudaError_t launch_append(const AppendParams& p, bool vec, bool f16, int splits, cudaStream_t stream) {
  const int qk = vec ? p.Dqk / 16 : p.Dqk - p.r.rot / 2, v = vec ? p.Dv / 16 : p.Dv;
  const long long blocks = row_blocks(p.T, qk > v ? qk : v);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return pick<AppendParams, AppendK>(p, vec, f16, dim3(static_cast<unsigned>(blocks), splits), stream);
}

}  // namespace attn
