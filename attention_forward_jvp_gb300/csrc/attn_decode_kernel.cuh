// Attention of one query token per sequence over a paged key-value cache.
//
// Mathematics: S = s q K^T, O = softmax(S) V, LSE, for the query heads of one
// key head together.  One pass over the keys with a running maximum m and
// sum l per head: P = exp2(S' - m), O <- O exp2(m_old - m) + P V,
// l <- l exp2(m_old - m) + sum(P), with S' = S log2(e).  m moves only when a
// score passes it by more than 8 (P then stays below 2^8), so that most steps
// need neither the maximum over the lanes nor the rescale; for fp16 storage m
// lies below the maximum and moves sooner (DecodeReference).  Parts of a
// sequence are joined by the same rule, whatever their m.
//
// What bounds it: memory.  Every key and value is read once and used by G
// query heads, G flops a byte; tcgen05's 64 or 128 rows would be padding but
// for G of them, and the trip through tensor memory latency.  mma.sync with
// the keys (for O: the value columns) as the 16 rows and the query heads as
// the 8 columns has no padding from G = 8 on.
//
//   S^T (16 keys x 8 heads)    = K (16 x Dqk) Q^T
//   O^T (Dv x 8 heads)        += V^T (Dv x 16 keys) P^T
//
// K and V^T come from shared memory by ldmatrix (V^T by its transposing
// form), Q^T stays in registers, P^T is turned from S^T's accumulator layout
// to the operand's by movmatrix.  NT groups of 8 heads share a key's loads.
//
// Layout of the work: the 16-key steps of all (sequence, key head) pairs form
// one list, cut into equal ranges, one for each resident warp, whatever the
// lengths.  A warp walks its range alone, unit after unit, with a ring of its
// own in shared memory that it fills by 16-byte asynchronous copies, row by
// row through the page table: no block-wide barrier until the end, where the
// warps of a CTA join what they hold of one unit in shared memory.  A unit
// that lies within a warp, or within what a CTA joins, is finished there;
// parts of the others go to the workspace and attn_decode_join joins them, in
// order.  Rows behind the sequence's end are filled with zeros, so that
// whatever a page holds there never enters a product.
#pragma once
#include "attn_paged_kernels.h"
#include "ptx.cuh"

namespace attn {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;  // 0: the 16 bytes are zeroed, nothing is read
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// 16 neighbouring tokens of a sequence, of which n are live.  Where pages hold
// a multiple of 16 tokens (`whole`) they lie in one page, from slot `slot` on;
// else lanes r and r + 16 have the page and slot of token r.
struct DecodePlace {
  int page, slot, n;
};
__device__ __forceinline__ DecodePlace decode_lookup(const DecodeParams& p, bool whole, const int* pages, int first,
                                                     int len) {
  DecodePlace x;
  const int key = whole ? first : first + (threadIdx.x & 15);
  x.n = len - first;
  x.page = x.slot = 0;
  if (key < len) {
    const int e = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
    x.slot = key - e * p.page_size;
    x.page = pages[e];
  }
  return x;
}
// Reports a page out of range (apart from the look-up, whose load is on its way)
__device__ __forceinline__ void decode_report(const DecodeParams& p, bool whole, const DecodePlace& x) {
  const int row = whole ? 0 : threadIdx.x & 15;
  if (row < x.n && static_cast<unsigned>(x.page) >= static_cast<unsigned>(p.n_pages)) *p.err = 1;
}
// Their rows of D elements (d of them real) of one pool, by a warp, into
// 128-byte swizzled rows PITCH bytes apart (64-element chunks CHUNK apart).
// Rows that are not live or have no page, and what is behind d, become zeros.
// An instruction moves whole rows, so that every request is for a full line:
// with 64 bytes of 8 rows to an instruction instead, the same traffic took 2
// to 5 % longer (64 sequences of up to 8192: 191 us for 186.5).
template <int D, int PITCH, int CHUNK>
__device__ __forceinline__ void copy_rows(const DecodeParams& p, bool whole, const DecodePlace& x,
                                          const uint16_t* head, const long long (&st)[3], int d, uint32_t to) {
  constexpr int L = D / 8 < 32 ? D / 8 : 32, R = 32 / L;  // lanes of a row, rows of an instruction
  const int lane = threadIdx.x & 31, lr = lane / L, c = lane % L;
  to += (c >> 3) * CHUNK + lr * PITCH + (((c & 7) ^ lr) << 4);
  const bool has = static_cast<unsigned>(x.page) < static_cast<unsigned>(p.n_pages);
  if (whole) {
    const int n = has && 8 * c < d ? x.n : 0;
    const uint16_t* from = head + x.page * st[0] + (x.slot + lr) * st[2] + 8 * c;
#pragma unroll
    for (int i = 0; i < 16; i += R) {
      const bool live = i + lr < n;
      cp_async16((to ^ ((i & 7) << 4)) + i * PITCH, live ? from : p.q, live);
      from += R * st[2];
    }
  } else {
    const unsigned rows = __ballot_sync(0xffffffffu, has && (lane & 15) < x.n) >> lr;
    const long long at = x.page * st[0] + x.slot * st[2];
#pragma unroll
    for (int i = 0; i < 16; i += R) {
      const long long row = __shfl_sync(0xffffffffu, at, i + lr);
      const bool live = (rows >> i & 1u) && 8 * c < d;
      cp_async16((to ^ ((i & 7) << 4)) + i * PITCH, live ? head + row + 8 * c : p.q, live);
    }
  }
}
// Arrive on `bar` when all copies that this thread has issued have landed
// (the barrier's count includes this arrival).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
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
// Where the reference m of the probabilities P = exp2(S' - m) lies: `below` the
// maximum when it moves, and it moves when a score is more than `room` above it.
// A bf16 part of P has fp32's exponents, so m is the maximum.  Parts in fp16 end
// at 2^-24, and at 65504: with m 11 below and 15 of room P goes up to 2^15, the
// largest probability of a part is 2^11 or more, and 2^-25, the most that its
// parts drop of any other, is 2^-36 of it.  (m at the maximum dropped 2^-25 of
// it: a key that outweighs a long even tail by 2^25 hid the tail from O, though
// not from l.)  What lies between the two is how far the maximum may rise
// without a rescale: 4 cost what 8 do where scores are N(0, 1.5^2) (64 heads,
// D 64, 32 sequences of 8192: 151.5 us for 151.2), and 4 % on tcgen05 where they
// are N(0, 3^2) (157.9 for 151.9); 2 cost as much at the former and 9 % there,
// and 8, with m 7 below, leave an even tail 16 times the error.
template <bool F16>
struct DecodeReference {
  static constexpr float below = F16 ? 11.f : 0.f, room = F16 ? 15.f : 8.f;
};
// x, y rounded to the operand type (hi) and what the rounding left (lo), each
// packed: hi + lo holds 16 bits of a probability in bf16; in fp16 it is off by at
// most 2^-23 of one above 2^-2, and by 2^-25 below.  Rounding P so costs the
// output nothing next to its own rounding.
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

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// a / b of whole numbers >= 0, b > 0
__device__ __forceinline__ int divide(int a, int b) { return static_cast<uint32_t>(a) / static_cast<uint32_t>(b); }
__device__ __forceinline__ long long divide(long long a, long long b) {
  return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// The list of steps cut into ranges: `total` steps over `ranges` ranges, one
// more for the first `extra` of them; and the place of this thread's range.
struct DecodeRange {
  long long total, ranges, each, extra;
  long long lo, cta_lo, cta_hi;  // first step of the range, of its CTA, behind the CTA's last
  int count;                     // steps of the range
  int b, hu, t, len;             // sequence, unit and step of lo, the sequence's length
  bool idle;                     // some sequence may be empty
  __device__ long long start(long long x) const { return x < ranges ? each * x + (x < extra ? x : extra) : total; }
  // the range that step x falls to
  __device__ long long owner(long long x) const {
    return x < extra * (each + 1) ? divide(x, each + 1) : extra + divide(x - extra * (each + 1), each);
  }
};
struct DecodeWords {
  int* lens;          // [threads]
  uint32_t* sums;     // [threads]
  long long* totals;  // [2][warps]
};

// Thread x holds sequence x (and adds up those behind it, a block's width
// apart): its length, and the steps up to it within its warp.  I: int where
// no list of this shape can pass 2^31 steps, else long long.  BN: keys of a
// step; NW: warps of a CTA, which has a range for each of them or one.
template <class I, int BN, int NW, bool PER_WARP>
__device__ __forceinline__ DecodeRange decode_plan(const DecodeParams& p, const DecodeWords& s) {
  constexpr int THREADS = NW * 32;
  constexpr unsigned ALL = 0xffffffffu;
  constexpr int R = PER_WARP ? NW : 1;  // ranges of a CTA
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const I HU = p.Hkv * p.chunks;
  auto length = [&](int b, bool& odd) {
    const int n = p.seq_lens[b];
    odd = odd || n < 0 || n > p.capacity;
    return n < 0 ? 0 : (n > p.capacity ? p.capacity : n);
  };
  auto scan = [&](I x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const I y = __shfl_up_sync(ALL, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  bool odd = false;
  int n = tid < p.B ? length(tid, odd) : 0;
  I inc = scan((n + BN - 1) / BN), rest = 0;
  if (p.B > THREADS) {
    for (int b = tid + THREADS; b < p.B; b += THREADS) rest += (length(b, odd) + BN - 1) / BN;
#pragma unroll
    for (int o = 16; o; o >>= 1) rest += __shfl_xor_sync(ALL, rest, o);
  }
  if (odd && blockIdx.x == 0) *p.err = 1;
  // (a sum within a warp fits 32 bits: 32 sequences of at most 2^26 steps)
  s.lens[tid] = n;
  s.sums[tid] = static_cast<uint32_t>(inc);
  if (lane == 31) s.totals[warp] = inc;
  if (lane == 0) s.totals[NW + warp] = rest;
  const bool idle = __syncthreads_or((tid < p.B && n == 0) || p.B > THREADS);
  I cum = scan(lane < NW ? static_cast<I>(s.totals[lane]) : 0);  // steps up to warp `lane`
  I steps = __shfl_sync(ALL, cum, NW - 1);
  if (p.B > THREADS) {
    I r = lane < NW ? static_cast<I>(s.totals[NW + lane]) : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) r += __shfl_xor_sync(ALL, r, o);
    steps += r;
  }
  const I total = steps * HU, most = static_cast<I>(gridDim.x) * R;
  I ranges = (total >> kDecodeMinStepsLog) + 1;
  ranges = ranges > most ? most : ranges;
  ranges = ranges > total ? total : ranges;
  ranges = ranges < 1 ? 1 : ranges;
  DecodeRange w;
  const I each = divide(total, ranges);
  w.idle = idle;
  w.total = total;
  w.ranges = ranges;
  w.each = each;
  w.extra = total - each * ranges;
  const int first = blockIdx.x * R, mine = first + (PER_WARP ? warp : 0);
  w.lo = w.start(mine);
  w.count = static_cast<int>(w.start(mine + 1) - w.lo);
  w.cta_lo = w.start(first);
  w.cta_hi = w.start(first + R);
  if (w.count == 0) w.lo = w.cta_lo;
  w.b = w.hu = w.t = w.len = 0;
  if (w.cta_lo >= total) return w;
  // the sequence: the first whose steps, with those before it, pass x; the
  // warps' places may lie in several blocks' widths of sequences
  const I x = divide(static_cast<I>(w.lo), HU);
  I base = 0;
  for (int b0 = 0;;) {
    const I all = __shfl_sync(ALL, cum, NW - 1);
    if (base <= x && x < base + all) {
      I y = x - base;
      const int chunk = __popc(__ballot_sync(ALL, lane < NW && cum <= y));
      if (chunk > 0) y -= __shfl_sync(ALL, cum, chunk - 1);
      const uint32_t v = s.sums[chunk * 32 + lane];
      const int k = __popc(__ballot_sync(ALL, v <= static_cast<uint32_t>(y)));
      if (k > 0) y -= __shfl_sync(ALL, v, k - 1);
      // y: place of x within the sequence's steps; in the list, each step
      // counts once for every unit
      w.b = b0 + chunk * 32 + k;
      w.len = s.lens[chunk * 32 + k];
      const int nt = (w.len + BN - 1) / BN;
      const I r = y * HU + (static_cast<I>(w.lo) - x * HU);
      const I hu = divide(r, static_cast<I>(nt));
      w.hu = static_cast<int>(hu);
      w.t = static_cast<int>(r - hu * nt);
    }
    base += all;
    b0 += THREADS;
    if (b0 >= p.B || w.cta_hi <= static_cast<long long>(base) * HU) break;
    n = b0 + tid < p.B ? length(b0 + tid, odd) : 0;
    inc = scan((n + BN - 1) / BN);
    __syncthreads();
    s.lens[tid] = n;
    s.sums[tid] = static_cast<uint32_t>(inc);
    if (lane == 31) s.totals[warp] = inc;
    __syncthreads();
    cum = scan(lane < NW ? static_cast<I>(s.totals[lane]) : 0);
  }
  return w;
}

// Sequences without keys: O = 0, LSE = -inf
static __device__ __noinline__ void decode_idle(const DecodeParams& p) {
  const int Hq = p.Hkv * p.G;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (p.seq_lens[b] > 0 && p.capacity > 0) continue;
    for (int i = threadIdx.x; i < Hq * (p.dv / 8); i += blockDim.x)
      reinterpret_cast<uint4*>(p.o + static_cast<long long>(b) * Hq * p.dv)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = threadIdx.x; i < Hq; i += blockDim.x) p.lse[static_cast<long long>(b) * Hq + i] = -INFINITY;
    if (p.by_unit)
      for (int i = threadIdx.x; i < p.Hkv * p.chunks; i += blockDim.x)
        p.desc[b * p.Hkv * p.chunks + i] = make_int4(-1, 0, 0, 0);
  }
}

// Where the parts of a unit are that begins in range x (of R to a CTA) and
// has its last step at `end`, in another range: in x's part 1; in part 0 of
// the first range of each CTA behind, that of the end included (z: how many
// CTAs lie between, -1 when the unit ends in x's own); and, where the range
// that it ends in goes on to another unit and is not that first one, in part
// 0 of that (w, else -1).  `desc` has this by units, with x before (-1: the
// unit is complete), or by ranges, with the unit before.
__device__ __forceinline__ void decode_complete(const DecodeParams& p, int b, int hu) {
  if (p.by_unit) p.desc[b * p.Hkv * p.chunks + hu] = make_int4(-1, 0, 0, 0);
}
template <int R>
__device__ __forceinline__ void decode_describe(const DecodeParams& p, const DecodeRange& w, int b, int hu, int x,
                                                long long end) {
  const int z = static_cast<int>(w.owner(end)), c = x / R, e = z / R;
  const bool own = w.start(z + 1LL) != end + 1 && (e == c || z != e * R);
  if (p.by_unit) p.desc[b * p.Hkv * p.chunks + hu] = make_int4(x, 0, e - c - 1, own ? z : -1);
  else p.desc[x] = make_int4(b, hu, e - c - 1, own ? z : -1);
}

// Eight warps with as many stages of 16 keys as shared memory holds (up to
// four), or four where it holds less than two, or more warps of a small head
// dim: a multiple of four always, since nine warps, three on one of the SM's
// four parts, were slower than eight (D 128: 198 us for 186).  Q stays in
// registers unless it and the accumulators would pass 176.
template <int DQ, int DV, int NT>
struct DecodePlan {
  static constexpr int BN = kDecodeBN;
  static constexpr int STAGE = BN * (DQ + DV) * 2;
  static constexpr int K_BYTES = BN * DQ * 2;
  static constexpr int ACC_REGS = DV / 4 * NT, Q_REGS = DQ / 8 * NT;
  static constexpr bool QREG = ACC_REGS + Q_REGS <= 176;
  static constexpr int Q_BYTES = QREG ? 0 : DQ / 16 * NT * 256;
  // words of the planning (8 bytes a thread, 16 a warp) and of the joining (a range and 24 a warp)
  static constexpr int MISC_BYTES = (8 * 32 + 16 + 24 + sizeof(DecodeRange)) * kDecodeMaxWarps;
  static constexpr int FIT = 226 * 1024 - MISC_BYTES;
  static constexpr int S8 = (FIT / 8 - Q_BYTES) / STAGE, S4 = (FIT / 4 - Q_BYTES) / STAGE;
  static constexpr int S = S8 >= 2 ? (STAGE <= 4096 ? 3 : (S8 > 4 ? 4 : S8)) : S4;
  static constexpr int WARP_BYTES = S * STAGE + Q_BYTES;
  static constexpr int REGS = ACC_REGS + (QREG ? Q_REGS : 0) + 72;
  static constexpr int NW_REGS = REGS <= 128 ? 16 : (REGS <= 160 ? 12 : 8);  // 128, 168, 255 registers a thread
  static constexpr int NW_SMEM = FIT / WARP_BYTES;
  static constexpr int NW = (NW_SMEM < NW_REGS ? NW_SMEM : NW_REGS) / 4 * 4;
  static_assert(NW <= kDecodeMaxWarps, "decode plan");
  static constexpr int SMEM = NW * WARP_BYTES + MISC_BYTES;
  // O of 8 heads on its way out, rows padded against bank conflicts
  static constexpr int PITCH = DV + 4;
  static_assert(NW >= 4 && S >= 2 && 8 * PITCH * 4 <= STAGE && NT * 8 * (PITCH * 4 + 8) <= S * STAGE, "decode plan");
};

// WHOLE: pages of a multiple of 16 tokens (a choice made in the loop instead
// costs what whole rows gain).
template <int DQ, int DV, bool F16, int NT, bool WHOLE>
__global__ void __launch_bounds__(DecodePlan<DQ, DV, NT>::NW * 32, 1)
    attn_decode_kernel(const __grid_constant__ DecodeParams p) {
  using P = DecodePlan<DQ, DV, NT>;
  constexpr int BN = P::BN, S = P::S, NW = P::NW, THREADS = NW * 32, PITCH = P::PITCH;
  constexpr int KPITCH = DQ * 2, VPITCH = DV * 2;
  extern __shared__ __align__(128) char decode_smem[];
  char* smem = decode_smem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  char* mine = smem + warp * P::WARP_BYTES;  // this warp's ring, then its Q
  const uint32_t ring = smem_u32(mine);
  uint2* qs = reinterpret_cast<uint2*>(mine + S * P::STAGE) + lane;
  char* misc = smem + NW * P::WARP_BYTES;
  const DecodeWords words{reinterpret_cast<int*>(misc), reinterpret_cast<uint32_t*>(misc) + THREADS,
                          reinterpret_cast<long long*>(misc + 8 * THREADS)};
  // of each warp at its end: its last unit, whether it begins there, whether
  // it goes on from the warp before; the unit's last step
  DecodeRange* ranges = reinterpret_cast<DecodeRange*>(misc + P::MISC_BYTES - (24 + sizeof(DecodeRange)) * kDecodeMaxWarps);
  int4* held = reinterpret_cast<int4*>(misc + P::MISC_BYTES - 24 * kDecodeMaxWarps);
  long long* held_end = reinterpret_cast<long long*>(misc + P::MISC_BYTES - 8 * kDecodeMaxWarps);
  const int HU = p.Hkv * p.chunks;  // units of a sequence

  griddep_wait();
  griddep_launch_dependents();

  auto length = [&](int b) {
    const int n = p.seq_lens[b];
    return n < 0 ? 0 : (n > p.capacity ? p.capacity : n);
  };
  auto steps_of = [](int len) { return (len + BN - 1) / BN; };
  struct Cursor {
    int b, hu, t, nt, len;
  };
  // the next step of the list (the caller knows that there is one)
  auto advance = [&](Cursor& a) {
    if (++a.t < a.nt) return;
    a.t = 0;
    if (++a.hu < HU) return;
    a.hu = 0;
    while (a.b + 1 < p.B) {
      ++a.b;
      a.len = length(a.b);
      a.nt = steps_of(a.len);
      if (a.nt > 0) break;
    }
  };
  const int mi = lane >> 3, l8 = lane & 7, g = lane >> 2, q4 = lane & 3;
  // where the tokens of a step lie, and its key head
  struct Place : DecodePlace {
    int h;
  };
  auto lookup = [&](const Cursor& a) -> Place {
    return {decode_lookup(p, WHOLE, p.page_table + a.b * p.table_stride, a.t * BN, a.len),
            p.chunks == 1 ? a.hu : a.hu / p.chunks};
  };

  // ---- this warp's range, and the places of its first steps, looked up all
  // at once
  const int first = blockIdx.x * NW;  // this CTA's first warp
  const int me = first + warp;
  DecodeRange w = p.wide ? decode_plan<long long, BN, NW, true>(p, words) : decode_plan<int, BN, NW, true>(p, words);
  const int count = w.count;
  Cursor cur{w.b, w.hu, w.t, steps_of(w.len), w.len};  // the step computed next
  Cursor ahead = cur;                                  // the step that `next` is of
  Place next, now[S - 1];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    if (j < count) {
      (j < S - 1 ? now[j < S - 1 ? j : 0] : next) = lookup(ahead);
      if (j + 1 < count && j + 1 < S) advance(ahead);
    }
  }

  if (w.idle) decode_idle(p);
  if (p.split && !p.by_unit && lane == 0) p.desc[me] = make_int4(-1, 0, 0, 0);
  if (w.cta_lo >= w.total) return;
  // (kept in shared memory while the steps need the registers)
  if (lane == 0) ranges[warp] = w;

  float acc[NT][DV / 16][4];
  float m[NT][2], l[NT][2];  // heads 2 q4, 2 q4 + 1 of each group
  uint32_t qr[P::QREG ? DQ / 16 : 1][NT][2];
  auto clear = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int d = 0; d < DV / 16; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][d][e] = 0.f;
    }
  };
  // Q^T of a unit as the product's second operand: pairs of neighbouring
  // elements of head g of each group
  auto load_q = [&](const Cursor& a) {
    const int h = a.hu / p.chunks, g0 = (a.hu - h * p.chunks) * p.rows, n_rows = min(p.rows, p.G - g0);
    const uint16_t* base = p.q + a.b * p.qs[0] + (static_cast<long long>(h) * p.G + g0) * p.qs[1];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool in = 8 * n + g < n_rows;
      const uint16_t* row = base + (in ? 8 * n + g : 0) * p.qs[1];
#pragma unroll
      for (int ks = 0; ks < DQ / 16; ++ks) {
        uint32_t v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = 16 * ks + 8 * e + 2 * q4;
          v[e] = in && d < p.dqk ? *reinterpret_cast<const uint32_t*>(row + d) : 0u;
        }
        if constexpr (P::QREG) {
          qr[ks][n][0] = v[0];
          qr[ks][n][1] = v[1];
        } else {
          qs[(ks * NT + n) * 32] = make_uint2(v[0], v[1]);  // read back by this lane alone
        }
      }
    }
  };
  // O of group n to [head][Dv] in shared memory, scaled by f[head of the lane]
  auto spill = [&](float* to, int n, float f0, float f1) {
#pragma unroll
    for (int d = 0; d < DV / 16; ++d) {
      float* x = to + 2 * q4 * PITCH + 16 * d + g;
      x[0] = acc[n][d][0] * f0;
      x[PITCH] = acc[n][d][1] * f1;
      x[8] = acc[n][d][2] * f0;
      x[PITCH + 8] = acc[n][d][3] * f1;
    }
  };
  // four columns of a row that is complete
  auto write_row = [&](long long row, int col, float4 o, float mm, float ll) {
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    if (col < p.dv)
      *reinterpret_cast<uint2*>(p.o + row * p.dv + col) =
          make_uint2(pack2<F16>(o.x * inv, o.y * inv), pack2<F16>(o.z * inv, o.w * inv));
    if (col == 0) p.lse[row] = ll == 0.f ? -INFINITY : mm * 0.6931471805599453f + logf(ll);
  };

  clear();
  if (count > 0) {
    auto issue = [&](const Place& x, int stage) {
      const uint32_t to = ring + stage * P::STAGE;
      decode_report(p, WHOLE, x);
      copy_rows<DQ, KPITCH, 128>(p, WHOLE, x, p.k + x.h * p.kp[1], p.kp, p.dqk, to);
      copy_rows<DV, VPITCH, 128>(p, WHOLE, x, p.v + x.h * p.vp[1], p.vp, p.dv, to + P::K_BYTES);
    };
    load_q(cur);
#pragma unroll
    for (int j = 0; j < S - 1; ++j) {
      if (j < count) issue(now[j], j);
      cp_async_commit();
    }

    int t0 = cur.t;  // first step of the unit in this warp
    int stage = 0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      // refill the stage of the step before this one, which every lane has read
      __syncwarp();
      if (i + S - 1 < count) {
        issue(next, stage == 0 ? S - 1 : stage - 1);
        if (i + S < count) {
          advance(ahead);
          next = lookup(ahead);
        }
      }
      cp_async_commit();
      cp_async_wait<S - 1>();
      __syncwarp();

      const uint32_t sk = ring + stage * P::STAGE, sv = sk + P::K_BYTES;
      const int live = cur.len - cur.t * BN;  // keys of this step
      constexpr int CH = NT == 1 ? 2 : 1;     // chains of products
      float s[CH][NT][4];
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[c][n][e] = 0.f;
      const uint32_t k_row = sk + ((mi & 1) * 8 + l8) * KPITCH;
#pragma unroll
      for (int ks = 0; ks < DQ / 16; ++ks) {
        uint32_t ka[4];
        ldsm4(ka, k_row + (((2 * ks + (mi >> 1)) ^ l8) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (P::QREG) {
            mma16816<F16>(s[ks % CH][n], ka, qr[ks][n][0], qr[ks][n][1]);
          } else {
            const uint2 q = qs[(ks * NT + n) * 32];
            mma16816<F16>(s[ks % CH][n], ka, q.x, q.y);
          }
        }
      }
      bool grows = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (CH == 2) s[0][n][e] += s[1][n][e];
          s[0][n][e] *= p.scale_log2;
          if (g + (e >> 1) * 8 >= live) s[0][n][e] = -INFINITY;
          grows = grows || s[0][n][e] > m[n][e & 1] + DecodeReference<F16>::room;
        }
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[0][n][e], s[0][n][2 + e]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x = fmaxf(x - DecodeReference<F16>::below, m[n][e]);
            const float a = exp2_fast(m[n][e] - (x == -INFINITY ? 0.f : x));
            m[n][e] = x;
            l[n][e] *= a;
#pragma unroll
            for (int d = 0; d < DV / 16; ++d) {
              acc[n][d][e] *= a;
              acc[n][d][2 + e] *= a;
            }
          }
      }
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // a head whose scores are all -inf keeps weights of 0
        const float u0 = m[n][0] == -INFINITY ? 0.f : m[n][0], u1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float a = exp2_fast(s[0][n][2 * e] - u0), b = exp2_fast(s[0][n][2 * e + 1] - u1);
          l[n][0] += a;
          l[n][1] += b;
          split2<F16>(a, b, ph[n][e], pl[n][e]);
          ph[n][e] = movmatrix_t(ph[n][e]);
          pl[n][e] = movmatrix_t(pl[n][e]);
        }
      }
      const uint32_t v_row = sv + ((mi >> 1) * 8 + l8) * VPITCH;
#pragma unroll
      for (int d = 0; d < DV / 16; ++d) {
        uint32_t va[4];
        ldsm4t(va, v_row + (((2 * d + (mi & 1)) ^ l8) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816<F16>(acc[n][d], va, ph[n][0], ph[n][1]);
          mma16816<F16>(acc[n][d], va, pl[n][0], pl[n][1]);
        }
      }

      // ---- the unit ends here, or the range does
      const bool last = i + 1 == count;
      if (cur.t + 1 == cur.nt || last) {
        const bool begins = t0 == 0;
        const int h = cur.hu / p.chunks, g0 = (cur.hu - h * p.chunks) * p.rows, n_rows = min(p.rows, p.G - g0);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
            l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
            l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
          }
        if (!last) {  // (the range's last unit is joined with the other warps' below; this one ends here)
          const long long part = 2LL * me;
          const long long row0 = (static_cast<long long>(cur.b) * p.Hkv + h) * p.G + g0;
          if (begins && lane == 0) decode_complete(p, cur.b, cur.hu);
          float* scratch = reinterpret_cast<float*>(mine + stage * P::STAGE);  // read; refilled in the next step
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            __syncwarp();
            spill(scratch, n, 1.f, 1.f);
            __syncwarp();
#pragma unroll
            for (int x = lane; x < 8 * (DV / 4); x += 32) {
              const int r = x / (DV / 4), c4 = x % (DV / 4);
              const float ma = __shfl_sync(0xffffffffu, m[n][0], r >> 1), mb = __shfl_sync(0xffffffffu, m[n][1], r >> 1);
              const float la = __shfl_sync(0xffffffffu, l[n][0], r >> 1), lb = __shfl_sync(0xffffffffu, l[n][1], r >> 1);
              const float mm = r & 1 ? mb : ma, ll = r & 1 ? lb : la;
              const float4 o = *reinterpret_cast<const float4*>(scratch + r * PITCH + 4 * c4);
              const int row = 8 * n + r;
              if (row < n_rows) {
                if (begins) {
                  write_row(row0 + row, 4 * c4, o, mm, ll);
                } else {
                  *reinterpret_cast<float4*>(p.part_o + (part * p.rows + row) * DV + 4 * c4) = o;
                  if (c4 == 0) p.part_ml[part * p.rows + row] = make_float2(mm, ll);
                }
              }
            }
          }
        }
        if (last) {
          if (lane == 0) {
            // goes on where the warp before has left off?
            const bool goes_on = warp > 0 && i == cur.t - t0 && t0 > 0;
            held[warp] = make_int4(cur.b, cur.hu, begins ? 1 : 0, goes_on ? 1 : 0);
            held_end[warp] = ranges[warp].lo + i + (cur.nt - 1 - cur.t);
          }
        } else {
          clear();
          advance(cur);
          t0 = 0;
          load_q(cur);
        }
      } else {
        ++cur.t;
      }
      stage = stage + 1 == S ? 0 : stage + 1;
    }
  }

  // ---- what the warps hold of their last units: joined, written
  constexpr int ROWS = NT * 8;
  float* parts = reinterpret_cast<float*>(mine);
  float2* my_ml = reinterpret_cast<float2*>(parts + ROWS * PITCH);  // behind O
  cp_async_wait<0>();
  __syncwarp();
  if (count > 0) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      spill(parts + 8 * n * PITCH, n, 1.f, 1.f);
      if (g == 0) {
        my_ml[8 * n + 2 * q4] = make_float2(m[n][0], l[n][0]);
        my_ml[8 * n + 2 * q4 + 1] = make_float2(m[n][1], l[n][1]);
      }
    }
  }
  __syncthreads();
  w = ranges[warp];
  // groups of warps with parts of one unit, by their first warps
  const int used = static_cast<int>(min(static_cast<long long>(NW), w.ranges - first));  // warps with steps
  const unsigned leads = __ballot_sync(0xffffffffu, lane < used && held[lane < used ? lane : 0].w == 0);
  const int items = p.rows * (DV / 4);
#pragma unroll 1
  for (int y = tid; y < __popc(leads) * items; y += THREADS) {
    const int gi = y / items, r = (y - gi * items) / (DV / 4), c4 = y % (DV / 4);
    unsigned left = leads;
    for (int k = 0; k < gi; ++k) left &= left - 1;
    const int w0 = __ffs(left) - 1;
    left &= left - 1;
    const int w1 = left ? __ffs(left) - 1 : used;
    const int4 u = held[w0];
    const long long end = held_end[w0];  // the unit's last step
    const bool begins = u.z != 0, ends = end < w.start(first + w1);
    const int h = p.chunks == 1 ? u.y : u.y / p.chunks, g0 = (u.y - h * p.chunks) * p.rows;
    if (r >= min(p.rows, p.G - g0)) continue;
    const long long part = 2LL * (first + w0) + (begins ? 1 : 0);
    float mm = -INFINITY, ll = 0.f;
    for (int x = w0; x < w1; ++x)
      mm = fmaxf(mm, reinterpret_cast<const float2*>(smem + x * P::WARP_BYTES + ROWS * PITCH * 4)[r].x);
    const float top = mm == -INFINITY ? 0.f : mm;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = w0; x < w1; ++x) {
      const char* from = smem + x * P::WARP_BYTES;
      const float2 s = reinterpret_cast<const float2*>(from + ROWS * PITCH * 4)[r];
      const float f = exp2_fast(s.x - top);
      const float4 z = *reinterpret_cast<const float4*>(from + (r * PITCH + 4 * c4) * 4);
      ll = fmaf(f, s.y, ll);
      o.x = fmaf(f, z.x, o.x);
      o.y = fmaf(f, z.y, o.y);
      o.z = fmaf(f, z.z, o.z);
      o.w = fmaf(f, z.w, o.w);
    }
    if (begins && ends) {
      write_row((static_cast<long long>(u.x) * p.Hkv + h) * p.G + g0 + r, 4 * c4, o, mm, ll);
      if (r == 0 && c4 == 0) decode_complete(p, u.x, u.y);
    } else {
      *reinterpret_cast<float4*>(p.part_o + (part * p.rows + r) * DV + 4 * c4) = o;
      if (c4 == 0) p.part_ml[part * p.rows + r] = make_float2(mm, ll);
      if (r == 0 && c4 == 0 && begins) decode_describe<NW>(p, w, u.x, u.y, first + w0, end);
    }
  }
}

// Joins the parts of the units that several ranges of the kernels above share:
// block (c, y) takes some heads (the y-th part of them) of unit c, or, where
// there are more units than CTAs, of those that begin in CTA c and end in
// another range.  A warp takes a head of one unit,
// or its parts together with other warps when there are fewer heads than
// warps; U parts' rows are on their way at a time.
constexpr int kJoinWarps = 8;

template <int DV, bool F16>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_decode_join(const __grid_constant__ DecodeParams p) {
  constexpr int NW = kJoinWarps, VPL = DV / 32;  // values of a lane
  constexpr int U = VPL > 4 ? 4 : 8;             // parts on their way
  constexpr unsigned ALL = 0xffffffffu;
  __shared__ float sum[NW][DV];
  __shared__ float2 stat[NW];
  __shared__ int4 units[kDecodeMaxWarps];
  __shared__ int from[kDecodeMaxWarps];
  __shared__ int n_units;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cw = p.cta_warps;
  const int r0 = blockIdx.y * p.join_rows, rows = min(p.join_rows, p.rows - r0);
  griddep_wait();
  griddep_launch_dependents();
  if (p.by_unit) {
    if (threadIdx.x == 0) {
      const int4 d = p.desc[blockIdx.x];
      const int hu = p.Hkv * p.chunks, b = blockIdx.x / hu;
      // (a wait that ran out of time may have left it unwritten)
      const bool sound = d.x >= 0 && d.x < p.ranges && d.z >= -1 && d.z + 1 < p.ranges / cw - d.x / cw && d.w >= -1 &&
                         d.w < p.ranges;
      units[0] = make_int4(b, blockIdx.x - b * hu, d.z, d.w);
      from[0] = d.x;
      n_units = sound ? 1 : 0;
    }
  } else if (warp == 0) {
    int4 d = make_int4(-1, 0, 0, 0);
    if (lane < cw) d = p.desc[blockIdx.x * cw + lane];
    const unsigned have = __ballot_sync(ALL, d.x >= 0);
    if (d.x >= 0) {
      const int at = __popc(have & ((1u << lane) - 1));
      units[at] = d;
      from[at] = blockIdx.x * cw + lane;
    }
    if (lane == 0) n_units = __popc(have);
  }
  __syncthreads();
  const int items = n_units * rows;
  int sh = 0;  // log2 of the warps of an item
  while (items << (sh + 1) <= NW && sh < 3) ++sh;
  for (int i0 = 0; i0 < items; i0 += NW >> sh) {
    const int it = i0 + (warp >> sh), s = warp & ((1 << sh) - 1);
    bool on = it < items;
    const int u = on ? it / rows : 0, r = on ? r0 + it - u * rows : 0;
    const int4 d = units[u];
    const int h = p.chunks == 1 ? d.y : d.y / p.chunks, g0 = (d.y - h * p.chunks) * p.rows;
    on = on && g0 + r < p.G;  // (the last units of a key head may have fewer)
    // parts, in order (decode_describe)
    const int parts = d.z + 2 + (d.w >= 0 ? 1 : 0), c0 = on ? from[u] / cw : 0;
    auto row_of = [&](int i) {
      const int w = i == 0 ? from[u] : (i <= d.z + 1 ? (c0 + i) * cw : d.w);
      return (2 * w + (i == 0 ? 1 : 0)) * p.rows + r;
    };
    float m = -INFINITY, l = 0.f, acc[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc[v] = 0.f;
    // adds a part: fa scales what is held, fb the part
    auto add = [&](float mb, float lb, const float (&y)[VPL]) {
      const float n = fmaxf(m, mb), top = n == -INFINITY ? 0.f : n;
      const float fa = exp2_fast(m - top), fb = exp2_fast(mb - top);
      m = n;
      l = l * fa + lb * fb;
#pragma unroll
      for (int v = 0; v < VPL; ++v) acc[v] = acc[v] * fa + y[v] * fb;
    };
    if (on) {
#pragma unroll 1
      for (int k0 = s; k0 < parts; k0 += U << sh) {
        float y[U][VPL];
        float2 st[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int at = row_of(min(k0 + (j << sh), parts - 1));
          st[j] = p.part_ml[at];
          const float* z = p.part_o + static_cast<long long>(at) * DV + lane * VPL;
#pragma unroll
          for (int v = 0; v < VPL; v += 2) {
            const float2 x = *reinterpret_cast<const float2*>(z + v);
            y[j][v] = x.x;
            y[j][v + 1] = x.y;
          }
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
          if (k0 + (j << sh) < parts) add(st[j].x, st[j].y, y[j]);
      }
    }
    if (sh > 0) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) sum[warp][lane * VPL + v] = acc[v];
      if (lane == 0) stat[warp] = make_float2(m, l);
      __syncthreads();
    }
    if (on && s == 0) {
      for (int k = 1; k < 1 << sh; ++k) {
        float y[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) y[v] = sum[warp + k][lane * VPL + v];
        add(stat[warp + k].x, stat[warp + k].y, y);
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const long long row = (static_cast<long long>(d.x) * p.Hkv + h) * p.G + g0 + r;
#pragma unroll
      for (int v = 0; v < VPL; v += 2)
        if (lane * VPL + v < p.dv)
          *reinterpret_cast<uint32_t*>(p.o + row * p.dv + lane * VPL + v) =
              pack2<F16>(acc[v] * inv, acc[v + 1] * inv);
      if (lane == 0) p.lse[row] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
    }
    if (sh > 0) __syncthreads();
  }
}

template <class K>
cudaError_t decode_launch_one(K kernel, const DecodeParams& p, dim3 grid, int threads, int smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
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

// Blocks of the join: about two an SM, which are resident at a time (eight for
// each CTA, most of them without a unit, took four rounds: 32 sequences of
// 8192, D 128, 8 heads 95.7 us for 90, 64 heads 118 for 109).
inline void plan_join(DecodeParams& p, int ctas) {
  const long long units = static_cast<long long>(p.B) * p.Hkv * p.chunks;
  p.ranges = ctas * p.cta_warps;
  p.by_unit = p.split && units <= ctas ? 1 : 0;
  const int blocks = 2 * ctas / static_cast<int>(p.by_unit ? units : ctas);  // for the heads of a unit
  p.join_rows = (p.rows + blocks - 1) / blocks;
}
template <int DV, bool F16>
cudaError_t launch_join(const DecodeParams& p, int ctas, cudaStream_t stream) {
  const dim3 grid(p.by_unit ? p.B * p.Hkv * p.chunks : ctas, (p.rows + p.join_rows - 1) / p.join_rows);
  return decode_launch_one(attn_decode_join<DV, F16>, p, grid, kJoinWarps * 32, 0, stream);
}

template <int DQ, int DV, bool F16, int NT, bool WHOLE>
cudaError_t launch_decode_nt(DecodeParams& p, int ctas, cudaStream_t stream) {
  using P = DecodePlan<DQ, DV, NT>;
  static bool attr_done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    e = cudaFuncSetAttribute(attn_decode_kernel<DQ, DV, F16, NT, WHOLE>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM);
    if (e != cudaSuccess) return e;
    // the same division of the SM's memory as the kernel before it: changing
    // it would have to wait for the SM to drain
    e = cudaFuncSetAttribute(attn_decode_join<DV, F16>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  p.cta_warps = P::NW;
  plan_join(p, ctas);
  e = decode_launch_one(attn_decode_kernel<DQ, DV, F16, NT, WHOLE>, p, dim3(ctas), P::NW * 32, P::SMEM, stream);
  if (e != cudaSuccess || !p.split) return e;
  return launch_join<DV, F16>(p, ctas, stream);
}

}  // namespace attn
