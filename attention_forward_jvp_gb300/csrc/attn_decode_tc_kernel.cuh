// The paged decode for many query heads on a key head (more than
// decode_warp_rows: 9 to 33 and more, by the head dims): the same list of
// steps, ranges and joining as attn_decode_kernel.cuh, with 64-key tiles, a
// range for each CTA, and the products on tcgen05.
//
//   S (128 x 64)   = Q K^T       Q: the unit's heads as rows, from shared memory
//   O (128 x Dv)  += P V         P: from tensor memory, V as it lies (MN-major)
//
// What has to bound it is memory, up to 128 heads: at D 128 an SM's share of
// the bandwidth brings a tile in 1400 cycles, and the tensor core multiplies it
// in 770 whatever the heads (lanes short of 128 are unused).  On mma.sync every
// 8 heads' columns would read the tile from shared memory again (64 heads, Dqk
// 256, Dv 128: 140 us; here 80).
//
// Warps 0-7 are the softmax: two to a quadrant of 32 lanes (32 heads), each
// with half of a tile's columns; quadrants behind the last head do nothing.
// Up to 64 heads stand twice in Q, as rows 0-63 and 64-127: the first two
// quadrants take the even tiles and the others the odd ones (the rows of P
// that are not a quadrant's stay zero), each with a running maximum, sum and
// O of its own, joined at the unit's end.  (32 sequences of 8192 keys, 64
// heads, D 64: 203 us with every quadrant at every tile, 169 so; 154 since
// copies move whole rows.)
// Warps 8-11 bring tiles (16 keys each) by 16-byte asynchronous copies, row by
// row through the page table; a tile's barrier counts the copies in as they
// land.  The last warp issues the products: S of tile i + 1 before O of tile
// i.  That lane is what bounds the kernel where memory does not (D 128, 64
// heads: 1700 cycles a tile): the products, those of O twice because P comes
// in two parts, and three waits.
// Both head dims 256: only two tiles fit beside Q, so keys and values have a
// ring each (a key stage is free again as soon as S is, a tile and a softmax
// before the values') and two groups of four warps bring the even and the odd
// tiles: 115 -> 101 us at 24 heads (95 since).  At D 128 the second barrier
// of a tile and the registers of the second group cost more than they give
// (112 -> 120 us).
// S and P have two buffers each in tensor memory.  P is split into two
// 16-bit parts there, like the warps' P of the other kernel.
#pragma once
#include "attn_decode_kernel.cuh"
#include "attn_kernel.cuh"

namespace attn {

constexpr int kTcBN = 64, kTcRows = 128;

// Whether the phase of `bar` with this parity is complete, without waiting
// (mbar_try_wait may suspend the thread for a while).
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The wait for 16 registers' loads from tensor memory.
__device__ __forceinline__ void tmem_wait_ld16_regs(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]) :: "memory");
}

template <int DQ, int DV>
struct DecodeTcPlan {
  static constexpr int SUB = kTcBN * 128;                // 64 columns of a tile
  static constexpr int K_TILE = DQ / 64 * SUB, V_TILE = DV / 64 * SUB, TILE = K_TILE + V_TILE;
  // a ring and barriers of their own for keys and values, two groups of
  // producers; else a tile's keys and values share a stage's barriers
  static constexpr bool SPLIT = TILE > 48 * 1024;
  static constexpr int GROUPS = SPLIT ? 2 : 1, ISSUER = 8 + 4 * GROUPS, NW = ISSUER + 1, THREADS = NW * 32;
  static constexpr int Q_SUB = kTcRows * 128, Q_TILE = DQ / 64 * Q_SUB;
  // words of the planning, sums and maxima of two units, O on its way from
  // the odd tiles' rows to the even ones' (16 columns of each half), barriers
  static constexpr int SUMS = 2 * 3 * kTcRows * 4, SWAP = 2 * 64 * 16 * 4, CTL = 512;
  static constexpr int MISC = 8 * THREADS + 16 * NW + SUMS + SWAP + CTL;
  static constexpr int FIT = 227 * 1024 - MISC - 1024;   // (1024: alignment)
  static constexpr int NQ = !SPLIT && 2 * Q_TILE + 3 * TILE <= FIT ? 2 : 1;
  static constexpr int S_FIT = (FIT - NQ * Q_TILE) / TILE, S = S_FIT > 8 ? 8 : S_FIT;  // stages
  static constexpr int OFF_K = NQ * Q_TILE, OFF_V = OFF_K + S * K_TILE, OFF_MISC = OFF_V + S * V_TILE;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;
  // barriers
  static constexpr int B_KF = 0, B_KE = S, B_VF = SPLIT ? 2 * S : B_KF, B_VE = SPLIT ? 3 * S : B_KE, B_SF = 4 * S,
                       B_PF = B_SF + 2, B_QE = B_SF + 4, B_OF = B_SF + 6, B_OE = B_SF + 7, B_LS = B_SF + 8,
                       B_XF = B_SF + 9, B_XE = B_SF + 10, B_DRAIN = B_SF + 11, NBAR = B_SF + 12;
  // tensor memory columns: S, S, P, P (upper | lower parts), O
  static constexpr int COL_P = 128, COL_O = 256, TMEM = 512;
  static_assert(S >= 2 && NBAR * 8 <= CTL - 16, "decode plan");
  // the stages of a group are its own, whose phases it sees one by one
  static_assert(S % GROUPS == 0, "decode plan");
};

template <int DQ, int DV, bool F16>
__global__ void __launch_bounds__(DecodeTcPlan<DQ, DV>::THREADS, 1)
    attn_decode_tc_kernel(const __grid_constant__ DecodeParams p) {
  using P = DecodeTcPlan<DQ, DV>;
  constexpr int BN = kTcBN, S = P::S, NQ = P::NQ;
  extern __shared__ __align__(128) char decode_smem[];
  char* smem = decode_smem + ((1024 - (smem_u32(decode_smem) & 1023)) & 1023);  // swizzle atoms of 1024 bytes
  const uint32_t base = smem_u32(smem);
  char* misc = smem + P::OFF_MISC;
  const DecodeWords words{reinterpret_cast<int*>(misc), reinterpret_cast<uint32_t*>(misc) + P::THREADS,
                          reinterpret_cast<long long*>(misc + 8 * P::THREADS)};
  float* sums = reinterpret_cast<float*>(misc + 8 * P::THREADS + 16 * P::NW);  // [2 units][l, l, m][row]
  float* swap = sums + P::SUMS / 4;                                            // [2 halves][16 columns][row]
  char* ctl = misc + P::MISC - P::CTL;
  const uint32_t bar0 = smem_u32(ctl);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(ctl + P::CTL - 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + P::CTL - 12);
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int HU = p.Hkv * p.chunks;
  const int quads = (p.rows + 31) / 32;  // quadrants with heads
  const int copies = quads <= 2 ? 2 : 1;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(bar(P::B_KF + i), 128);
      mbar_init(bar(P::B_KE + i), 1);
      if (P::SPLIT) {
        mbar_init(bar(P::B_VF + i), 128);
        mbar_init(bar(P::B_VE + i), 1);
      }
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(P::B_SF + i), 1);
      mbar_init(bar(P::B_PF + i), 2 * quads);
      mbar_init(bar(P::B_QE + i), 1);
    }
    mbar_init(bar(P::B_OF), 1);
    mbar_init(bar(P::B_OE), 2 * quads * copies);
    mbar_init(bar(P::B_LS), 64 * quads * copies);
    mbar_init(bar(P::B_XF), 64 * quads);
    mbar_init(bar(P::B_XE), 64 * quads);
    mbar_init(bar(P::B_DRAIN), 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == P::ISSUER) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), P::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  griddep_wait();
  griddep_launch_dependents();
  // (barriers and the tensor-memory address are published by its barrier)
  const DecodeRange w =
      p.wide ? decode_plan<long long, BN, P::NW>(p, words, 1, 0) : decode_plan<int, BN, P::NW>(p, words, 1, 0);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int count = w.count;
  if (copies == 2) {
    // each quadrant's rows of the other parity's P, which stay zero
    if (warp < 8) {
      const uint32_t z[32] = {};
      tmem_st_32x32b_x32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + P::COL_P +
                             ((warp & 2) ? 0 : 64) + (warp >> 2) * 32, z);
      tmem_wait_st();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (w.idle) decode_idle(p);
  if (p.split && !p.by_unit && tid == 0) p.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);

  const Waiter W{abort_flag, p.err + 1, p.timeout_ns};
  auto wait_all = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait_bar(bar(b), parity, W)); };
  auto wait_sleep = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait_bar_sleep(bar(b), parity, W)); };
  auto length = [&](int b) {
    const int n = p.seq_lens[b];
    return n < 0 ? 0 : (n > p.capacity ? p.capacity : n);
  };
  auto steps_of = [](int len) { return (len + BN - 1) / BN; };
  struct Cursor {
    int b, hu, t, nt, len;
  };
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
  Cursor cur{w.b, w.hu, w.t, steps_of(w.len), w.len};
  auto unit = [&](const Cursor& a, int& h, int& g0, int& n_rows) {
    h = p.chunks == 1 ? a.hu : a.hu / p.chunks;
    g0 = (a.hu - h * p.chunks) * p.rows;
    n_rows = min(p.rows, p.G - g0);
  };

  if (warp >= 8 && warp < P::ISSUER && count > 0) {
    // ------------------------------------------------------------ producers
    const int k0 = (warp & 3) * 16;  // this warp's rows of a tile
    const uint16_t *kh = nullptr, *vh = nullptr;  // of the unit's key head
    const int* pages = nullptr;                   // of the sequence
    auto enter = [&](const Cursor& a) {
      const int h = p.chunks == 1 ? a.hu : a.hu / p.chunks;
      kh = p.k + h * p.kp[1];
      vh = p.v + h * p.vp[1];
      pages = p.page_table + a.b * p.table_stride;
    };
    auto lookup = [&](const Cursor& a) { return decode_lookup(p, p.whole, pages, a.t * BN + k0, a.len); };
    // the unit's heads; rows behind them, up to the quadrant's end, are zeros
    auto issue_q = [&](const Cursor& a, int qb) {
      int h, g0, n_rows;
      unit(a, h, g0, n_rows);
      const uint16_t* q = p.q + a.b * p.qs[0] + (static_cast<long long>(h) * p.G + g0) * p.qs[1];
      const uint32_t qd = base + qb * P::Q_TILE;
      constexpr int PIECES = DQ / 8;
      for (int x = tid & 127; x < quads * 32 * PIECES; x += 128) {
        const int r = x / PIECES, c = x % PIECES;
        const bool in = r < n_rows && 8 * c < p.dqk;
        const uint32_t to = qd + (c >> 3) * P::Q_SUB + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        const uint16_t* from = in ? q + r * p.qs[1] + 8 * c : p.q;
        cp_async16(to, from, in);
        if (copies == 2) cp_async16(to + 64 * 128, from, in);
      }
    };
    // Every tile, or every second one.  A thread's arrival counts it in when
    // its copies so far have landed; the warp that issues the products makes
    // them visible to the tensor core.
    bool ok = true;
    const int group = (warp - 8) >> 2;
    int j = group, seg = 0;  // (cur: tile j, of unit seg in this CTA)
    int stage = j;
    uint32_t phase = 1, q_phase = 0;
    auto step = [&]() {
      advance(cur);
      if (cur.t == 0) ++seg;
    };
    if (j == 1 && count > 1) step();
    enter(cur);
    DecodePlace next = lookup(cur);
    while (j < count) {
      ok = wait_all(P::B_KE + stage, phase);
      if (!ok) break;
      if (j == 0 || cur.t == 0) {
        // (two groups: the one buffer's barrier of the group that is to fill
        // it next, which so sees every phase of its own)
        if (P::GROUPS == 1) {
          ok = wait_all(P::B_QE + seg % NQ, ((seg / NQ) & 1u) ^ 1u);
        } else if (j > 0) {
          ok = wait_all(P::B_QE + group, q_phase);
          q_phase ^= 1u;
        }
        if (!ok) break;
        issue_q(cur, seg % NQ);
      }
      decode_report(p, p.whole, next);
      copy_rows<DQ, 128, P::SUB>(p, p.whole, next, kh, p.kp, p.dqk, base + P::OFF_K + stage * P::K_TILE + k0 * 128);
      // (the failure-detection hook: the first tile never arrives)
      const bool arrives = j > 0 || !p.skip_first_load || blockIdx.x != 0;
      if (P::SPLIT) {
        if (arrives) cp_async_arrive(bar(P::B_KF + stage));
        ok = wait_all(P::B_VE + stage, phase);
        if (!ok) break;
      }
      copy_rows<DV, 128, P::SUB>(p, p.whole, next, vh, p.vp, p.dv, base + P::OFF_V + stage * P::V_TILE + k0 * 128);
      if (P::SPLIT || arrives) cp_async_arrive(bar(P::B_VF + stage));
      j += P::GROUPS;
      if (j >= count) break;
      stage += P::GROUPS;
      if (stage >= S) {
        stage -= S;
        phase ^= 1u;
      }
      const int was = seg;
      step();
      if (P::GROUPS == 2) step();
      if (seg != was) enter(cur);
      next = lookup(cur);
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == P::ISSUER && count > 0) {
    // -------------------------------------------------------------- products
    // One lane alone: its waits and issues are the longest chain of a tile,
    // and votes between them would lengthen it.
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc_16(kTcRows, BN, false, F16), idesc_o = idesc_16(kTcRows, DV, true, F16);
      constexpr uint32_t kHi = sdesc_hi_sw128(1024);
      const uint32_t lo_q = sdesc_lo(base, 16), lo_k = sdesc_lo(base + P::OFF_K, 16);
      const uint32_t lo_v = sdesc_lo(base + P::OFF_V, P::SUB);
      bool ok = true;
      int seg = 0, pv_seg = 0;
      bool first = true;                       // of its unit in this CTA: the tile whose O is next
      int ks = 0, vs = 0;                      // stages of the tiles whose S and O are next
      uint32_t kp = 0, vp = 0;
      // O of tile j, the last of its unit or not
      auto products_o = [&](int j, bool last) {
        ok = wait_bar(bar(P::B_PF + (j & 1)), (j >> 1) & 1u, W);
        // the first product of a unit overwrites O: the unit before has left it
        if (ok && first) ok = wait_bar(bar(P::B_OE), (pv_seg & 1u) ^ 1u, W);
        if (P::SPLIT && ok) ok = wait_bar(bar(P::B_VF + vs), vp, W);
        if (!ok) return;
        if (P::SPLIT) fence_proxy_async_smem();
        tc_fence_after();
        const uint32_t a = tmem + P::COL_P + (j & 1) * 64, v = lo_v + vs * (P::V_TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) {
          const uint64_t d = sdesc_join(v + ((kk * 2048) >> 4), kHi);
          mma_ts(tmem + P::COL_O, a + 8 * kk, d, idesc_o, first && kk == 0 ? 0u : 1u);
          mma_ts(tmem + P::COL_O, a + 32 + 8 * kk, d, idesc_o, 1u);
        }
        tc_commit(bar(P::B_VE + vs));
        if (last) tc_commit(bar(P::B_OF));
        first = last;
        pv_seg += last ? 1 : 0;
        if (++vs == S) {
          vs = 0;
          vp ^= 1u;
        }
      };
      // 1: barrier a has completed; 2: barrier b has, and a not yet; 0:
      // neither in time (the wait that follows reports it)
      auto wait_first = [&](uint32_t a, uint32_t pa, uint32_t b, uint32_t pb) {
        uint64_t t0 = 0;
        for (uint32_t it = 0;; ++it) {
          if (mbar_test_wait(a, pa)) return 1;
          if (mbar_test_wait(b, pb)) return 2;
          if ((it & 7u) != 7u) continue;
          if (t0 == 0) t0 = globaltimer_ns();
          else if (*abort_flag != 0 || globaltimer_ns() - t0 > p.timeout_ns) return 0;
        }
      };
      bool pending = false, last_before = false;  // O of tile i - 1
      for (int i = 0; ok && i < count; ++i) {
        const bool last = cur.t + 1 == cur.nt || i + 1 == count;
        // S of this tile before O of the one before, unless that is ready first
        const int which =
            pending ? wait_first(bar(P::B_KF + ks), kp, bar(P::B_PF + ((i - 1) & 1)), ((i - 1) >> 1) & 1u) : 0;
        if (which == 2) {
          products_o(i - 1, last_before);
          pending = false;
          if (!ok) break;
        }
        if (which != 1) ok = wait_bar(bar(P::B_KF + ks), kp, W);
        if (!ok) break;
        fence_proxy_async_smem();  // the copies, made by the generic proxy, before the products read them
        tc_fence_after();
        const uint32_t q = lo_q + (seg % NQ) * (P::Q_TILE >> 4), k = lo_k + ks * (P::K_TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < DQ / 16; ++kk) {
          const uint32_t oq = ((kk >> 2) * P::Q_SUB + (kk & 3) * 32) >> 4, ok_ = ((kk >> 2) * P::SUB + (kk & 3) * 32) >> 4;
          mma_ss(tmem + (i & 1) * BN, sdesc_join(q + oq, kHi), sdesc_join(k + ok_, kHi), idesc_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(bar(P::B_SF + (i & 1)));
        if (P::SPLIT) tc_commit(bar(P::B_KE + ks));
        if (last) {
          tc_commit(bar(P::B_QE + (P::GROUPS == 1 ? seg % NQ : (i + 1) & 1)));
          ++seg;
        }
        if (++ks == S) {
          ks = 0;
          kp ^= 1u;
        }
        if (pending) products_o(i - 1, last_before);
        pending = true;
        last_before = last;
        if (i + 1 < count) advance(cur);
      }
      if (ok && pending) products_o(count - 1, last_before);
      tc_commit(bar(P::B_DRAIN));
      drain_bar(bar(P::B_DRAIN), 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp < 8 && (copies == 2 ? (warp & 1) : (warp & 3)) < quads && count > 0) {
    // --------------------------------------------------------------- softmax
    const int quad = warp & 3, half = warp >> 2, lrow = quad * 32 + lane;
    const int odd = copies == 2 ? quad >> 1 : 0;  // takes the tiles of this parity
    const int row = lrow - 64 * odd;              // head
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    constexpr int DH = DV / 2;  // this warp's columns of O
    float m = -INFINITY, l = 0.f;
    bool ok = true, first = true;
    int seg = 0, t0 = cur.t;
    uint32_t swaps = 0;
    for (int i = 0; i < count; ++i) {
      const bool ends = cur.t + 1 == cur.nt, last = ends || i + 1 == count;
      if (copies == 1 || (i & 1) == odd) {
        ok = wait_sleep(P::B_SF + (i & 1), (i >> 1) & 1u);
        if (!ok) break;
        tc_fence_after();
        uint32_t x0[32], x1[32];  // this half's columns, the other's
        tmem_ld_32x32b_x32(tl + (i & 1) * BN + half * 32, x0);
        tmem_ld_32x32b_x32(tl + (i & 1) * BN + (half ^ 1) * 32, x1);
        tmem_wait_ld_regs(x0);
        tmem_regs_ready(x1);
        const int live = cur.len - cur.t * BN;
        if (live < BN) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (half * 32 + c >= live) x0[c] = 0xff800000u;
            if ((half ^ 1) * 32 + c >= live) x1[c] = 0xff800000u;
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 32; ++c) top = max3f(top, __uint_as_float(x0[c]), __uint_as_float(x1[c]));
        top *= p.scale_log2;
        if (__any_sync(0xffffffffu, top > m + DecodeReference<F16>::room)) {
          const float n = fmaxf(m, top - DecodeReference<F16>::below), a = exp2_fast(m - (n == -INFINITY ? 0.f : n));
          m = n;
          l *= a;
          if (!first) {
            // O is at rest once the products of the tile before are done
            ok = wait_sleep(P::B_VE + (i - 1) % S, ((i - 1) / S) & 1u);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < DH; c0 += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(tl + P::COL_O + half * DH + c0, o);
              tmem_wait_ld_regs(o);
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * a);
              tmem_st_32x32b_x32(tl + P::COL_O + half * DH + c0, o);
            }
            tmem_wait_st();
          }
        }
        const float u = m == -INFINITY ? 0.f : m;
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float a = exp2_fast(fmaf(__uint_as_float(x0[c]), p.scale_log2, -u));
          const float b = exp2_fast(fmaf(__uint_as_float(x0[c + 1]), p.scale_log2, -u));
          l += a + b;
          split2<F16>(a, b, hi[c / 2], lo[c / 2]);
        }
        const uint32_t tp = tl + P::COL_P + (i & 1) * 64 + half * 16;
        tmem_st_32x32b_x16(tp, hi);
        tmem_st_32x32b_x16(tp + 32, lo);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(P::B_PF + (i & 1)));
        first = false;
      }

      if (last) {
        // ---- the unit's part in this CTA is complete
        int h, g0, n_rows;
        unit(cur, h, g0, n_rows);
        float* ls = sums + (seg & 1) * 3 * kTcRows;
        ls[half * kTcRows + lrow] = l;
        if (half == 0) ls[2 * kTcRows + lrow] = m;
        mbar_arrive(bar(P::B_LS));  // (a bounded wait, unlike a named barrier's)
        ok = wait_sleep(P::B_LS, seg & 1u) && wait_sleep(P::B_OF, seg & 1u);
        if (!ok) break;
        tc_fence_after();
        float sum = ls[lrow] + ls[kTcRows + lrow], mine = 1.f;  // of all tiles; the factor of this row's O
        if (copies == 2) {
          const int other = lrow ^ 64;
          const float mo = ls[2 * kTcRows + other], n = fmaxf(m, mo), top = n == -INFINITY ? 0.f : n;
          mine = exp2_fast(m - top);
          sum = sum * mine + (ls[other] + ls[kTcRows + other]) * exp2_fast(mo - top);
          m = n;
        }
        const bool begins = t0 == 0;
        const bool in = row < n_rows;
        const long long at = (static_cast<long long>(cur.b) * p.Hkv + h) * p.G + g0 + row;
        const long long part = (2LL * blockIdx.x + (begins ? 1 : 0)) * p.rows + row;
        const float inv = begins && ends ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
#pragma unroll 1
        for (int c0 = 0; c0 < DH; c0 += 16) {
          __syncwarp();  // rows of a quadrant behind the unit's heads have no part in the stores below
          uint32_t o[16];
          tmem_ld_32x32b_x16(tl + P::COL_O + half * DH + c0, o);
          tmem_wait_ld16_regs(o);
          if (copies == 2) {
            float* x = swap + half * 16 * 64 + row;
            if (odd) {
              ok = wait_sleep(P::B_XE, (swaps & 1u) ^ 1u);  // the columns before have been taken
              if (!ok) break;
#pragma unroll
              for (int c = 0; c < 16; ++c) x[c * 64] = __uint_as_float(o[c]) * mine;
              mbar_arrive(bar(P::B_XF));
            } else {
              ok = wait_sleep(P::B_XF, swaps & 1u);
              if (!ok) break;
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(fmaf(__uint_as_float(o[c]), mine, x[c * 64]));
              mbar_arrive(bar(P::B_XE));
            }
            ++swaps;
          }
          const int col = half * DH + c0;
          if (in && !odd) {
            if (begins && ends) {
#pragma unroll
              for (int c = 0; c < 16; c += 8) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  y[e] = pack2<F16>(__uint_as_float(o[c + 2 * e]) * inv, __uint_as_float(o[c + 2 * e + 1]) * inv);
                if (col + c < p.dv)
                  *reinterpret_cast<uint4*>(p.o + at * p.dv + col + c) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else {
#pragma unroll
              for (int c = 0; c < 16; c += 4)
                *reinterpret_cast<uint4*>(p.part_o + part * DV + col + c) =
                    make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
            }
          }
        }
        if (!ok) break;
        if (in && half == 0 && !odd) {
          if (begins && ends) p.lse[at] = sum == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(sum);
          else p.part_ml[part] = make_float2(m, sum);
        }
        if (begins && tid == 0) {
          if (ends) decode_complete(p, cur.b, cur.hu);
          else decode_describe(p, w, 1, cur.b, cur.hu, blockIdx.x, w.lo + i + (cur.nt - 1 - cur.t));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(P::B_OE));
        ++seg;
        first = true;
        m = -INFINITY;
        l = 0.f;
        t0 = 0;
      }
      if (i + 1 < count) advance(cur);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == P::ISSUER) tmem_dealloc(tmem, P::TMEM);
}

template <int DQ, int DV, bool F16>
cudaError_t launch_decode_tc(DecodeParams& p, int ctas, cudaStream_t stream) {
  using P = DecodeTcPlan<DQ, DV>;
  static bool attr_done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    e = cudaFuncSetAttribute(attn_decode_tc_kernel<DQ, DV, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attn_decode_join<DV, F16>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  p.cta_warps = 1;
  plan_join(p, ctas);
  e = decode_launch_one(attn_decode_tc_kernel<DQ, DV, F16>, p, dim3(ctas), P::THREADS, P::SMEM, stream);
  if (e != cudaSuccess || !p.split) return e;
  return launch_join<DV, F16>(p, ctas, stream);
}

template <int DQ, int DV, bool F16, int NT = 1>
cudaError_t launch_decode_warps(DecodeParams& p, int nt, int ctas, cudaStream_t stream) {
  if constexpr (8 * NT < decode_warp_rows(DQ, DV))
    if (nt > NT) return launch_decode_warps<DQ, DV, F16, NT + 1>(p, nt, ctas, stream);
  return p.whole ? launch_decode_nt<DQ, DV, F16, NT, true>(p, ctas, stream)
                 : launch_decode_nt<DQ, DV, F16, NT, false>(p, ctas, stream);
}

template <int DQ, int DV, bool F16>
cudaError_t launch_decode(DecodeParams& p, int nt, int ctas, cudaStream_t stream) {
  if (nt > 0) return launch_decode_warps<DQ, DV, F16>(p, nt, ctas, stream);
  return launch_decode_tc<DQ, DV, F16>(p, ctas, stream);
}

}  // namespace attn
