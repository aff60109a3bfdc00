// Attention of one query token per sequence over a paged key-value cache.
//
// Mathematics: S = s q K^T, O = softmax(S) V, LSE, for the G query heads of
// one key head together.  One pass over the keys with a running maximum m
// and sum l per row: P = exp2(S' - m), O <- O exp2(m_old - m) + P V,
// l <- l exp2(m_old - m) + rowsum(P), with S' = S log2(e).  Parts of a
// sequence are joined by the same rule.
//
// What bounds it: memory.  Every key and value is read once and used by G
// rows, 2 G flops a byte; at G <= 16 the 16-row mma.sync steps below need a
// sixth of their issue rate to keep up with memory, so the 128-row
// tcgen05 tiles (64 rows at least, all but G of them padding) and their
// trips through tensor memory would buy nothing here.
//
// Layout of the work: the 64-key tiles of all (sequence, key head) pairs
// form one list, cut into equal ranges, one for each resident CTA, whatever
// the lengths; a CTA walks its range, unit after unit.  A unit that lies
// within one CTA is finished there; parts of the others go to the workspace
// and attn_decode_join joins them, in order.  The warps of a CTA share a
// tile's keys (16 or 32 each) and, above 16 rows, its rows.
//
// Tiles come by 16-byte asynchronous copies, row by row through the page
// table, into a ring that keeps two to five tiles in flight; rows behind the
// sequence's end are filled with zeros, so that whatever a page holds there
// never enters a product.
#pragma once
#include "attn_paged_kernels.h"
#include "ptx.cuh"

namespace attn {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;  // 0: the 16 bytes are zeroed, nothing is read
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8)
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// x, y rounded to the operand type (hi) and what the rounding left (lo), each
// packed: hi + lo holds 16 or more bits of a probability, so that rounding P
// costs the output nothing next to its own rounding.
template <bool F16>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack2<F16>(x, y);
  float hx, hy;
  if constexpr (F16) {
    __half2 h;
    *reinterpret_cast<uint32_t*>(&h) = hi;
    const float2 f = __half22float2(h);
    hx = f.x;
    hy = f.y;
  } else {
    hx = bf16_lo(hi);
    hy = bf16_hi(hi);
  }
  lo = pack2<F16>(x - hx, y - hy);
}

constexpr int decode_pow2_floor(int x) {
  int r = 1;
  while (2 * r <= x) r *= 2;
  return r;
}

template <int DQ, int DV, int NW>
struct DecodePlan {
  static constexpr int BN = kDecodeBN;
  static constexpr int THREADS = NW * 32;
  static constexpr int CTAS = decode_ctas_per_sm(DQ, DV, NW);
  static constexpr int ROWS = NW == 4 ? 16 : kDecodeMaxRows;
  static constexpr int Q_BYTES = ROWS * DQ * 2;
  static constexpr int K_BYTES = BN * DQ * 2;
  static constexpr int TILE_BYTES = BN * (DQ + DV) * 2;
  // per-warp row statistics, scan words
  static constexpr int MISC_BYTES = NW * 16 * 8 + 256;
  // (the row table beside the ring: page and slot of each key in flight)
  static constexpr int BUDGET = (CTAS == 2 ? 113 : 226) * 1024 - Q_BYTES - MISC_BYTES;
  static constexpr int STAGES_FIT = BUDGET / (TILE_BYTES + BN * 8);
  static constexpr int STAGES = STAGES_FIT > 6 ? 6 : STAGES_FIT;
  static constexpr int TAB = STAGES;  // table entries: a tile's is free once its copies are issued
  static constexpr int SMEM = Q_BYTES + STAGES * TILE_BYTES + TAB * BN * 8 + MISC_BYTES;
  // columns of O that the warps exchange at a time through one stage
  static constexpr int CW_FIT = decode_pow2_floor(TILE_BYTES / (NW * 64));
  static constexpr int CW = CW_FIT < DV ? CW_FIT : DV;
  static_assert(STAGES >= 2 && CW >= 32, "decode plan");
};

template <int DQ, int DV, bool F16, int NW>
__global__ void __launch_bounds__(NW * 32, decode_ctas_per_sm(DQ, DV, NW))
    attn_decode_kernel(const __grid_constant__ DecodeParams p) {
  using P = DecodePlan<DQ, DV, NW>;
  constexpr int BN = P::BN, S = P::STAGES, THREADS = P::THREADS;
  constexpr int QPITCH = DQ * 2, KPITCH = DQ * 2, VPITCH = DV * 2;
  constexpr bool QREG = DQ <= 128;  // Q fragments stay in registers
  extern __shared__ __align__(128) char smem[];
  const uint32_t sq = smem_u32(smem);
  const uint32_t ring = sq + P::Q_BYTES;
  int2* tab = reinterpret_cast<int2*>(smem + P::Q_BYTES + S * P::TILE_BYTES);
  float2* ml = reinterpret_cast<float2*>(tab + P::TAB * BN);
  long long* scan = reinterpret_cast<long long*>(ml + NW * 16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int HU = p.Hkv * p.chunks;  // units of a sequence

  griddep_wait();
  griddep_launch_dependents();

  auto length = [&](int b) {
    const int n = __ldg(p.seq_lens + b);
    return n < 0 ? 0 : (n > p.capacity ? p.capacity : n);
  };
  auto tiles_of = [](int len) { return (len + BN - 1) / BN; };

  // ---- this CTA's range [lo, hi) of the tile list
  long long sum = 0;
  for (int b = tid; b < p.B; b += THREADS) {
    const int raw = __ldg(p.seq_lens + b), n = length(b);
    if (raw != n && blockIdx.x == 0) *p.err = 1;
    sum += tiles_of(n);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) scan[warp] = sum;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) total += scan[w];
  total *= HU;
  long long ctas = (total + p.min_tiles - 1) / p.min_tiles;
  if (ctas > gridDim.x) ctas = gridDim.x;
  const int c = blockIdx.x;
  const long long lo = c < ctas ? total * c / ctas : 0;
  const long long hi = c < ctas ? total * (c + 1) / ctas : 0;

  // ---- sequences without keys: O = 0, LSE = -inf
  for (int b = c; b < p.B; b += gridDim.x) {
    if (length(b) != 0) continue;
    const int Hq = p.Hkv * p.G;
    for (int i = tid; i < Hq * (p.dv / 8); i += THREADS)
      reinterpret_cast<uint4*>(p.o + static_cast<long long>(b) * Hq * p.dv)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < Hq; i += THREADS) p.lse[static_cast<long long>(b) * Hq + i] = -INFINITY;
  }
  if (p.split && tid == 0) p.desc[c] = make_int4(-1, 0, 0, 0);
  const int count = static_cast<int>(hi - lo);
  if (count == 0) return;

  // ---- the sequence that tile lo belongs to
  struct Cursor {
    int b, hu, t, nt, len;
  };
  Cursor cur;
  {
    long long before = 0;
    int b0 = 0;
    long long r = 0;
    for (;; b0 += THREADS) {  // ends: lo < total
      const int b = b0 + tid;
      const long long mine = b < p.B ? static_cast<long long>(tiles_of(length(b))) * HU : 0;
      long long inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      __syncthreads();
      if (lane == 31) scan[warp] = inc;
      if (tid == 0) scan[NW] = -1;
      __syncthreads();
      long long base = before, all = before;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        if (w < warp) base += scan[w];
        all += scan[w];
      }
      const long long start = base + inc - mine;
      if (mine > 0 && start <= lo && lo < start + mine) {
        scan[NW] = b;
        scan[NW + 1] = lo - start;
      }
      __syncthreads();
      if (scan[NW] >= 0) {
        cur.b = static_cast<int>(scan[NW]);
        r = scan[NW + 1];
        break;
      }
      if (b0 + THREADS >= p.B) return;  // (never: the lengths changed under the kernel)
      before = all;
    }
    cur.len = length(cur.b);
    cur.nt = max(tiles_of(cur.len), 1);
    cur.hu = static_cast<int>(r / cur.nt);
    cur.t = static_cast<int>(r - static_cast<long long>(cur.hu) * cur.nt);
  }
  // the next tile of the list; the caller knows that there is one
  auto advance = [&](Cursor& a) {
    if (++a.t < a.nt) return;
    a.t = 0;
    if (++a.hu < HU) return;
    a.hu = 0;
    do {
      ++a.b;
      a.len = length(a.b);
      a.nt = tiles_of(a.len);
    } while (a.nt == 0 && a.b + 1 < p.B);
  };

  // ---- page table look-ups, tiles ahead of the copies
  auto lookup = [&](const Cursor& a, int key_in_tile) -> int2 {
    const int key = a.t * BN + key_in_tile;
    if (key >= a.len) return make_int2(-1, 0);
    const int e = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
    const int slot = key - e * p.page_size;
    int page = __ldg(p.page_table + a.b * p.table_stride + e);
    if (page < 0 || page >= p.n_pages) {
      *p.err = 1;
      page = -1;
    }
    return make_int2(page, slot);
  };
  // ---- copies of one tile
  auto issue = [&](int hu, int stage, int entry) {
    const int h = hu / p.chunks;
    const int2* row = tab + entry * BN;
    constexpr int KC = DQ / 8, VC = DV / 8;  // 16-byte pieces of a row
    const uint32_t kd = ring + stage * P::TILE_BYTES, vd = kd + P::K_BYTES;
    {
      const int piece = tid % KC;
      const bool in = piece * 8 < p.dqk;
      const uint16_t* base = p.k + h * p.kp[1] + piece * 8;
#pragma unroll
      for (int r = tid / KC; r < BN; r += THREADS / KC) {
        const int2 e = row[r];
        const bool live = in && e.x >= 0;
        const uint16_t* src = live ? base + e.x * p.kp[0] + e.y * p.kp[2] : p.q;
        cp_async16(kd + r * KPITCH + ((piece ^ (r & 7)) << 4), src, live);
      }
    }
    {
      const int piece = tid % VC;
      const bool in = piece * 8 < p.dv;
      const uint16_t* base = p.v + h * p.vp[1] + piece * 8;
#pragma unroll
      for (int r = tid / VC; r < BN; r += THREADS / VC) {
        const int2 e = row[r];
        const bool live = in && e.x >= 0;
        const uint16_t* src = live ? base + e.x * p.vp[0] + e.y * p.vp[2] : p.q;
        cp_async16(vd + r * VPITCH + ((piece ^ (r & 7)) << 4), src, live);
      }
    }
  };
  // ---- query rows of a unit, 16-byte pieces
  constexpr int QC = DQ / 8;
  constexpr int QN = (P::ROWS * QC + THREADS - 1) / THREADS;  // pieces of a thread
  auto load_q = [&](const Cursor& a, uint4 (&reg)[QN]) {
    const int h = a.hu / p.chunks, chunk = a.hu - h * p.chunks;
    const int g0 = chunk * p.rows, n = min(p.rows, p.G - g0);
    const uint16_t* base = p.q + a.b * p.qs[0] + static_cast<long long>(h * p.G + g0) * p.qs[1];
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int x = tid + i * THREADS, r = x / QC, piece = x % QC;
      reg[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < n && piece * 8 < p.dqk) reg[i] = *reinterpret_cast<const uint4*>(base + r * p.qs[1] + piece * 8);
    }
  };
  auto store_q = [&](const uint4 (&reg)[QN]) {
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int x = tid + i * THREADS, r = x / QC, piece = x % QC;
      if (r < P::ROWS) *reinterpret_cast<uint4*>(smem + r * QPITCH + ((piece ^ (r & 7)) << 4)) = reg[i];
    }
  };

  Cursor ahead = cur;     // the tile whose page numbers are looked up next
  int looked = 0;         // tiles looked up
  int2 next_row;          // row `tid` of tile `looked`, on its way (tid < BN)
  // rows of the first S tiles at once
  {
    constexpr int GROUPS = THREADS / BN;
    int2 rows[(S + GROUPS - 1) / GROUPS];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      if (j < count) {
        if (tid / BN == j % GROUPS) rows[j / GROUPS] = lookup(ahead, tid % BN);
        if (j + 1 < count) advance(ahead);
        looked = j + 1;
      }
    }
#pragma unroll
    for (int j = 0; j < S; ++j)
      if (j < count && tid / BN == j % GROUPS) tab[j % P::TAB * BN + tid % BN] = rows[j / GROUPS];
  }
  uint4 qreg[QN];
  load_q(cur, qreg);
  store_q(qreg);
  __syncthreads();
  Cursor fill = cur;  // the tile whose copies are issued next
#pragma unroll
  for (int j = 0; j < S - 1; ++j) {
    if (j < count) {
      issue(fill.hu, j, j);
      if (j + 1 < count) advance(fill);
    }
    cp_async_commit();
  }
  if (tid < BN && looked < count) next_row = lookup(ahead, tid);

  // ---- accumulators
  const int wr = warp % p.wr, wk = warp / p.wr, WK = NW / p.wr;
  const int keys_w = BN / WK;  // keys of this warp in a tile
  const int mi = lane >> 3, l8 = lane & 7, g = lane >> 2, q4 = lane & 3;
  uint32_t qf[QREG ? DQ / 16 : 1][4];
  const uint32_t q_row = sq + (wr * 16 + (mi & 1) * 8 + l8) * QPITCH;
  auto q_frag = [&](int ks, uint32_t (&f)[4]) { ldsm4(f, q_row + (((ks * 2 + (mi >> 1)) ^ l8) << 4)); };
  float acc[DV / 8][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g and g + 8
#pragma unroll
  for (int i = 0; i < DV / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  if constexpr (QREG) {
#pragma unroll
    for (int ks = 0; ks < DQ / 16; ++ks) q_frag(ks, qf[ks]);
  }
  int seg_t0 = cur.t;  // first tile of the unit in this CTA

  int stage = 0;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    cp_async_wait<S - 2>();
    __syncthreads();
    // refill the stage of the tile before this one
    const int j = i + S - 1;
    if (j < count) {
      issue(fill.hu, stage == 0 ? S - 1 : stage - 1, j % P::TAB);
      if (j + 1 < count) advance(fill);
    }
    cp_async_commit();
    // rows of tile i + S: its entry was that of tile i, read S - 1 tiles ago
    if (looked < count) {
      if (tid < BN) tab[looked % P::TAB * BN + tid] = next_row;
      if (looked + 1 < count) {
        advance(ahead);
        if (tid < BN) next_row = lookup(ahead, tid);
      }
      ++looked;
    }

    const uint32_t sk = ring + stage * P::TILE_BYTES, sv = sk + P::K_BYTES;
    const int live = cur.len - cur.t * BN;  // keys of this tile
#pragma unroll 1
    for (int k0 = wk * keys_w; k0 < (wk + 1) * keys_w; k0 += 16) {
      if (k0 >= live) break;  // (warp-uniform)
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t k_row = sk + (k0 + (mi >> 1) * 8 + l8) * KPITCH;
#pragma unroll
      for (int ks = 0; ks < DQ / 16; ++ks) {
        uint32_t kb[4];
        ldsm4(kb, k_row + (((ks * 2 + (mi & 1)) ^ l8) << 4));
        if constexpr (QREG) {
          mma16816<F16>(s0, qf[ks], kb[0], kb[1]);
          mma16816<F16>(s1, qf[ks], kb[2], kb[3]);
        } else {
          uint32_t f[4];
          q_frag(ks, f);
          mma16816<F16>(s0, f, kb[0], kb[1]);
          mma16816<F16>(s1, f, kb[2], kb[3]);
        }
      }
      if (k0 + 16 > live) {
        const int k = k0 + 2 * q4;
        if (k >= live) s0[0] = s0[2] = -INFINITY;
        if (k + 1 >= live) s0[1] = s0[3] = -INFINITY;
        if (k + 8 >= live) s1[0] = s1[2] = -INFINITY;
        if (k + 9 >= live) s1[1] = s1[3] = -INFINITY;
      }
      float x0 = fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s1[0], s1[1]));
      float x1 = fmaxf(fmaxf(s0[2], s0[3]), fmaxf(s1[2], s1[3]));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
      const float n0 = fmaxf(m0, x0 * p.scale_log2), n1 = fmaxf(m1, x1 * p.scale_log2);
      // a row whose scores are all -inf keeps weights of 0
      const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
      if (__any_sync(0xffffffffu, n0 != m0 || n1 != m1)) {
        const float a0 = exp2_fast(m0 - u0), a1 = exp2_fast(m1 - u1);
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int d = 0; d < DV / 8; ++d) {
          acc[d][0] *= a0;
          acc[d][1] *= a0;
          acc[d][2] *= a1;
          acc[d][3] *= a1;
        }
        m0 = n0;
        m1 = n1;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s0[e] = exp2_fast(fmaf(s0[e], p.scale_log2, -u0));
        s1[e] = exp2_fast(fmaf(s1[e], p.scale_log2, -u0));
        s0[2 + e] = exp2_fast(fmaf(s0[2 + e], p.scale_log2, -u1));
        s1[2 + e] = exp2_fast(fmaf(s1[2 + e], p.scale_log2, -u1));
      }
      l0 += (s0[0] + s0[1]) + (s1[0] + s1[1]);
      l1 += (s0[2] + s0[3]) + (s1[2] + s1[3]);
      uint32_t ph[4], pl[4];
      split2<F16>(s0[0], s0[1], ph[0], pl[0]);
      split2<F16>(s0[2], s0[3], ph[1], pl[1]);
      split2<F16>(s1[0], s1[1], ph[2], pl[2]);
      split2<F16>(s1[2], s1[3], ph[3], pl[3]);
      const uint32_t v_row = sv + (k0 + (mi & 1) * 8 + l8) * VPITCH;
#pragma unroll
      for (int d = 0; d < DV / 16; ++d) {
        uint32_t vb[4];
        ldsm4t(vb, v_row + (((d * 2 + (mi >> 1)) ^ l8) << 4));
        mma16816<F16>(acc[2 * d], ph, vb[0], vb[1]);
        mma16816<F16>(acc[2 * d + 1], ph, vb[2], vb[3]);
        mma16816<F16>(acc[2 * d], pl, vb[0], vb[1]);
        mma16816<F16>(acc[2 * d + 1], pl, vb[2], vb[3]);
      }
    }

    // ---- end of the unit, or of the range: join the warps, write
    if (cur.t + 1 == cur.nt || i + 1 == count) {
      const Cursor done = cur;
      const bool more = i + 1 < count;
      if (more) {
        advance(cur);
        load_q(cur, qreg);
      }
      const bool begins = seg_t0 == 0, ends = done.t + 1 == done.nt;
      const int h = done.hu / p.chunks, chunk = done.hu - h * p.chunks;
      const int g0 = chunk * p.rows, n_rows = min(p.rows, p.G - g0);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      if (q4 == 0) {
        ml[warp * 16 + g] = make_float2(m0, l0);
        ml[warp * 16 + g + 8] = make_float2(m1, l1);
      }
      __syncthreads();  // statistics written; nobody reads this stage or Q any more
      if (more) store_q(qreg);
      // maximum and sum of row r of this CTA's part
      auto row_stat = [&](int r) -> float2 {
        const int w0 = r >> 4, rr = r & 15;
        float m = -INFINITY, l = 0.f;
        for (int w = 0; w < WK; ++w) m = fmaxf(m, ml[(w * p.wr + w0) * 16 + rr].x);
        const float u = m == -INFINITY ? 0.f : m;
        for (int w = 0; w < WK; ++w) {
          const float2 x = ml[(w * p.wr + w0) * 16 + rr];
          l += exp2_fast(x.x - u) * x.y;
        }
        return make_float2(m, l);
      };
      const float2 st0 = row_stat(wr * 16 + g), st1 = row_stat(wr * 16 + g + 8);
      const float f0 = exp2_fast(m0 - (st0.x == -INFINITY ? 0.f : st0.x));
      const float f1 = exp2_fast(m1 - (st1.x == -INFINITY ? 0.f : st1.x));
      const bool whole = begins && ends;
      const long long slot = 2LL * c + (begins ? 1 : 0);
      float* buf = reinterpret_cast<float*>(smem + P::Q_BYTES + stage * P::TILE_BYTES);
      constexpr int CW = P::CW, NB = CW / 8;  // 8-column blocks, swizzled by the row
      constexpr int SW = NB < 8 ? NB - 1 : 7;
#pragma unroll
      for (int c0 = 0; c0 < DV; c0 += CW) {
        if (c0 > 0) __syncthreads();
#pragma unroll
        for (int d = 0; d < NB; ++d) {
          float* x = buf + (warp * 16 + g) * CW + ((d ^ (g & SW)) * 8) + 2 * q4;
          const float* a = acc[c0 / 8 + d];
          *reinterpret_cast<float2*>(x) = make_float2(a[0] * f0, a[1] * f0);
          *reinterpret_cast<float2*>(x + 8 * CW) = make_float2(a[2] * f1, a[3] * f1);
        }
        __syncthreads();
        for (int x = tid; x < n_rows * (CW / 4); x += THREADS) {
          const int r = x / (CW / 4), c4 = x % (CW / 4);
          const int w0 = r >> 4, rr = r & 15;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int w = 0; w < WK; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(
                buf + ((w * p.wr + w0) * 16 + rr) * CW + (((c4 >> 1) ^ (rr & SW)) * 8) + (c4 & 1) * 4);
            o.x += y.x;
            o.y += y.y;
            o.z += y.z;
            o.w += y.w;
          }
          const int col = c0 + 4 * c4;
          if (whole) {
            const float2 st = row_stat(r);
            const float inv = st.y == 0.f ? 0.f : 1.f / st.y;
            const long long row = (static_cast<long long>(done.b) * p.Hkv + h) * p.G + g0 + r;
            if (col < p.dv)
              *reinterpret_cast<uint2*>(p.o + row * p.dv + col) =
                  make_uint2(pack2<F16>(o.x * inv, o.y * inv), pack2<F16>(o.z * inv, o.w * inv));
            if (col == 0) p.lse[row] = st.y == 0.f ? -INFINITY : st.x * 0.6931471805599453f + logf(st.y);
          } else {
            *reinterpret_cast<float4*>(p.part_o + (slot * p.rows + r) * DV + col) = o;
            if (col == 0) p.part_ml[slot * p.rows + r] = row_stat(r);
          }
        }
      }
      if (begins && !ends && tid == 0) {
        // the CTA that the unit's last tile falls to
        const long long last = lo + i + (done.nt - 1 - done.t);
        const int parts = static_cast<int>(((last + 1) * ctas - 1) / total) - c + 1;
        p.desc[c] = make_int4(done.b, done.hu, parts, 0);
      }
      if (more) {
        seg_t0 = 0;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
#pragma unroll
        for (int d = 0; d < DV / 8; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[d][e] = 0.f;
        // (store_q is ordered before this by the barriers of the exchange)
        if constexpr (QREG) {
#pragma unroll
          for (int ks = 0; ks < DQ / 16; ++ks) q_frag(ks, qf[ks]);
        }
      }
    } else {
      ++cur.t;
    }
    stage = stage + 1 == S ? 0 : stage + 1;
  }
}

// Joins the parts of a unit that several CTAs of the kernel above share:
// block c takes the unit that starts in CTA c and ends in a later one, if
// there is one.  A warp takes a row, or a row's parts together with other
// warps when there are fewer rows than warps.
template <int DV, bool F16>
__global__ void __launch_bounds__(512) attn_decode_join(const __grid_constant__ DecodeParams p) {
  constexpr int NW = 16, VPL = DV / 32;  // values of a lane
  __shared__ float part[NW][DV];
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x;
  const int4 d = p.desc[c];
  if (d.x < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = d.y / p.chunks, chunk = d.y - h * p.chunks;
  const int g0 = chunk * p.rows, n_rows = min(p.rows, p.G - g0);
  const int per_row = n_rows >= NW ? 1 : NW / n_rows;  // warps of a row
  const int parts = d.z;
  auto slot = [&](int i) { return 2LL * (c + i) + (i == 0 ? 1 : 0); };
  for (int r0 = 0; r0 < n_rows; r0 += NW / per_row) {
    const int r = r0 + warp / per_row, s = warp % per_row;
    const bool on = warp < NW / per_row * per_row && r < n_rows;
    float m = -INFINITY, l = 0.f, acc[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc[v] = 0.f;
    if (on) {
      for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.part_ml[slot(i) * p.rows + r].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float u = m == -INFINITY ? 0.f : m;
      for (int i = lane; i < parts; i += 32) {
        const float2 x = p.part_ml[slot(i) * p.rows + r];
        l += exp2_fast(x.x - u) * x.y;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll 4
      for (int i = s; i < parts; i += per_row) {
        const float w = exp2_fast(p.part_ml[slot(i) * p.rows + r].x - u);
        const float* x = p.part_o + (slot(i) * p.rows + r) * DV + lane * VPL;
#pragma unroll
        for (int v = 0; v < VPL; v += 2) {
          const float2 y = *reinterpret_cast<const float2*>(x + v);
          acc[v] = fmaf(w, y.x, acc[v]);
          acc[v + 1] = fmaf(w, y.y, acc[v + 1]);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) part[warp][lane * VPL + v] = acc[v];
    __syncthreads();
    if (on && s == 0) {
      for (int k = 1; k < per_row; ++k)
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] += part[warp + k][lane * VPL + v];
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const long long row = (static_cast<long long>(d.x) * p.Hkv + h) * p.G + g0 + r;
#pragma unroll
      for (int v = 0; v < VPL; v += 2)
        if (lane * VPL + v < p.dv)
          *reinterpret_cast<uint32_t*>(p.o + row * p.dv + lane * VPL + v) =
              pack2<F16>(acc[v] * inv, acc[v + 1] * inv);
      if (lane == 0) p.lse[row] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
    }
    __syncthreads();
  }
}

template <class K>
cudaError_t decode_launch_one(K kernel, const DecodeParams& p, int grid, int threads, int smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int DQ, int DV, bool F16, int NW>
cudaError_t launch_decode_nw(const DecodeParams& p, int ctas, cudaStream_t stream) {
  constexpr int smem = DecodePlan<DQ, DV, NW>::SMEM;
  static bool attr_done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    e = cudaFuncSetAttribute(attn_decode_kernel<DQ, DV, F16, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  e = decode_launch_one(attn_decode_kernel<DQ, DV, F16, NW>, p, ctas, NW * 32, smem, stream);
  if (e != cudaSuccess || !p.split) return e;
  return decode_launch_one(attn_decode_join<DV, F16>, p, ctas, 512, 0, stream);
}

template <int DQ, int DV, bool F16>
cudaError_t launch_decode(const DecodeParams& p, int nw, int ctas, cudaStream_t stream) {
  return nw == 4 ? launch_decode_nw<DQ, DV, F16, 4>(p, ctas, stream) : launch_decode_nw<DQ, DV, F16, 8>(p, ctas, stream);
}

}  // namespace attn
