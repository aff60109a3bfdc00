// The cache in 4 bits, reading back, weights and eviction: what the host side
// (attn_paged_cache.cu) hands to the kernels.
#pragma once
#include "attn_paged_kernels.h"

namespace attn {

// groups of a row of d elements that share a step and a least value
__host__ __device__ constexpr int groups4(int d) { return d < 64 ? 1 : d / 64; }

// Keys or values of a cache in 4 bits, by (page, head, token)
struct Pool4 {
  uint8_t* codes;
  uint16_t* scales;  // fp16: a row's steps, then its least values
  long long st[3];   // bytes
  long long ss[3];   // elements
};

// The pools of a 16-bit cache are in `a`; those of one in 4 bits here
struct Append4Params {
  AppendParams a;
  Pool4 k, v;
};

struct GatherParams {
  const uint16_t *k16, *v16;  // 16 bits
  long long kp[3], vp[3];
  Pool4 k, v;                 // 4 bits
  uint16_t *k_out, *v_out;
  long long ko[2], vo[2];     // head, token
  int Hkv, Dqk, Dv;
  int heads_per_split;
  long long T;
  const int* offsets;
  const int* page_table;
  long long table_stride;
  const int* seq_lens;
  int B, max_pages, n_pages, page_size;
  int* err;
};

cudaError_t launch_append4(const Append4Params& p, bool vec, bool f16, int splits, cudaStream_t stream);
// bits: 16 or 4; f16: the type that 4 bits become; wide: rows on 32-byte boundaries
cudaError_t launch_gather(const GatherParams& p, int bits, bool f16, bool wide, int splits, cudaStream_t stream);

// ------------------------------------------------------------------ decode
constexpr int kDecode4BN = 32;  // keys of a step

// Query heads of a warp at most, for G on a key head, in groups of 8: a second
// group shares the making of operands with the first and takes registers from
// it, so that fewer warps are resident.  More heads go to more warps, which walk
// over the same steps at the same time.  16 sequences of up to 32768 on two key
// heads, one group a warp and two (us): 256/256, 16 heads 91 and 123; 256/128 64
// and 70, with 32 heads 111 and 99; 64/64 41.5 and 39.4, with 32 heads 64 and 58
// (four groups).
constexpr int decode4_rows(int dv, int G) { return dv == 256 || (dv == 128 && G <= 16) ? 8 : 16; }

struct Decode4Params {
  DecodeParams d;  // (its 16-bit pools unused; Hkv, G, rows, chunks by the launch)
  Pool4 k, v;
  int narrow;      // copy_tokens4
  int sub_rows;    // query heads of a warp
  // set by the launch: warps of a range, each with heads of its own; the key
  // heads that they are of, 1 or all different
  int subs, heads;
};

// The decode kernel over a cache in 4 bits for kernel head dims DQ, DV and nt (1, 2)
// groups of 8 query heads to a unit, followed, when p.d.split, by the join
template <int DQ, int DV, bool F16>
cudaError_t launch_decode4(Decode4Params& p, int nt, int ctas, cudaStream_t stream);

// ----------------------------------------------------------------- weights
struct WeightParams {
  DecodeParams d;     // (no values, workspace or outputs)
  Pool4 k;            // of a cache in 4 bits
  int narrow;         // copy_tokens4
  int subs;           // set by the launch: warps of a range, each with a key head of its own
  int f16;            // the type of q
  float scale;        // of the scores
  const float* lse;   // [B, Hkv * G]
  const float* w;     // or null
  float* out;
  long long ws[2], os[2];  // sequence, head
  float decay;
  long long places;   // of a row
};
// dq: kernel head dim; bits: 16 or 4
cudaError_t launch_weights(const WeightParams& p, int dq, int bits, int ctas, cudaStream_t stream);

// ---------------------------------------------------------------- eviction
struct EvictParams {
  int B, Hkv, max_pages, n_pages, page_size, n_new;
  int capacity, new_capacity;  // keys of a row of the old table, of the new pages
  const int* page_table;
  long long table_stride;
  const int* seq_lens;
  const int* keep;             // or null
  int keep_all, sinks, recent;
  const int* pages;
  long long pages_stride;
  int* table_out;
  long long table_out_stride;
  int* lens_out;
  const float* w;
  float* w_out;
  long long ws[2], wos[2], places;
  int page_shift;              // log2 of page_size, or -1
  int2* index;                 // [B][Hkv][new_capacity]: page and slot of a head's kept tokens
  uint16_t *k16, *v16;
  long long kp[3], vp[3];
  Pool4 k, v;
  int Dqk, Dv;
  int* err;
};
// launches: how many kernels it came to
cudaError_t launch_evict(const EvictParams& p, int bits, int sms, cudaStream_t stream, int* launches);

}  // namespace attn
