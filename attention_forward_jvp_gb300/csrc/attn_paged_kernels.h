// Rotary positions and the paged cache: what the host side (attn_paged.cu)
// hands to the kernels (attn_rope.cu, attn_decode_kernel.cuh).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace attn {

// ------------------------------------------------------------- rope, append
struct RopeSpec {
  const unsigned long long* steps;  // turn per position, 2^64 = a full turn
  int rot;                          // rotated elements of a head (0: none)
  int interleaved;
  float scale;
  int inverse;
};

struct RopeTensor {
  const uint16_t* x;
  uint16_t* y;
  long long xs[3], ys[3];  // batch, head, token
  int H;
};

constexpr int kRopeTensors = 4;
constexpr int kRopeUnroll = 2;  // heads of a thread in flight

struct RopeParams {
  RopeTensor t[kRopeTensors];
  RopeSpec r;
  int n_tensors, heads;      // heads: of all tensors together
  int heads_per_split;       // heads of one blockIdx.y
  int D;
  long long N, rows;         // tokens of a batch entry, of all
  const int* positions;      // or null
  long long ps[2];
  const int* offsets;        // or null
  int n_seq;
};

struct AppendParams {
  RopeSpec r;
  const uint16_t *k, *v, *q;
  uint16_t *k_pool, *v_pool, *q_out;
  long long ks[2], vs[2], qs[2], qos[2];  // token, head
  long long kp[3], vp[3];                 // page, head, token
  int Hq, Hkv, Dqk, Dv;                   // Hq = 0: no queries
  int heads_per_split;
  long long T;
  const int* offsets;                     // or null: token b is of sequence b
  const int* page_table;
  long long table_stride;
  const int* seq_lens;
  int B, max_pages, n_pages, page_size;
  int* err;
};

// vec: every row 16-byte aligned, head dims and rotated width multiples of 16
cudaError_t launch_rope(const RopeParams& p, bool vec, bool f16, int splits, cudaStream_t stream);
cudaError_t launch_append(const AppendParams& p, bool vec, bool f16, int splits, cudaStream_t stream);

// -------------------------------------------------------------------- decode
constexpr int kDecodeBN = 16;        // keys of a step
// A list of n steps is cut into n / 2 + 1 ranges at most: most take two steps,
// and one or two of a list that is cut so finely take one (n / 2 ranges would
// leave a third step to one of them where n is odd).
constexpr int kDecodeMinStepsLog = 1;
constexpr int kDecodeMaxWarps = 16;  // warps of a CTA, at most
// Query heads of a unit that a warp takes at most, in groups of 8; more go to
// tcgen05.  Every group is another pass of mma.sync over a step and takes
// registers by the head dims, so the limit falls with them.  On either side of
// it, the warps' kernel and tcgen05 with one head more (32 sequences of 8192,
// us): 64/64 123 and 151, 128/64 107 and 112 at 32; 256/64 90 and 95, 64/128 96
// and 107, 128/128 99 and 101 at 24; 256/128 75 and 74, 64/256 93 and 91 at 16.
// (One group more: 256/128 93 for 82 at 24; 256/256 135 for 100 at 16.)
constexpr int decode_warp_rows(int dq, int dv) {
  return dv == 64 ? (dq <= 128 ? 32 : 24) : (dv == 128 ? (dq <= 128 ? 24 : 16) : (dq < 256 ? 16 : 8));
}
constexpr int kDecodeMaxRows = 128;   // query heads of a unit, at most

struct DecodeParams {
  const uint16_t *q, *k, *v;
  long long qs[2];             // sequence, head
  long long kp[3], vp[3];      // page, head, token
  const int* page_table;
  long long table_stride;
  const int* seq_lens;
  int B, n_pages, page_size, page_shift;  // page_shift: log2, or -1
  int capacity;                // keys a table row can hold
  int Hkv, G;                  // key heads, query heads of each
  int rows, chunks;            // query heads of a work unit, units of a key head
  int dqk, dv;                 // true head dims (<= the kernel's)
  int whole;                   // 1: pages hold a multiple of 16 tokens
  float scale_log2;
  uint16_t* o;
  float* lse;
  int4* desc;                  // by range, or by unit: the unit that starts in it and ends in a later one
  float2* part_ml;             // [warp][2][rows]
  float* part_o;               // [warp][2][rows][kernel Dv]
  int* err;                    // [0]: bad page or length, [1]: a wait timed out
  int split;                   // 0: no sequence can have more than one step
  unsigned long long timeout_ns;  // of a wait between the warps of a CTA (err[1])
  int skip_first_load;         // failure-detection hook
  int wide;                    // 1: the list of steps might pass 2^31
  // set by the launch: ranges of a CTA, of all; whether `desc` and the joining blocks go
  // by units; heads of a joining block
  int cta_warps, ranges, by_unit, join_rows;
};

// The decode kernel for kernel head dims DQ, DV and nt groups of 8 query heads
// to a unit, or (0) more of them than the warps' kernel takes, followed, when p.split, by the
// joining kernel.
template <int DQ, int DV, bool F16>
cudaError_t launch_decode(DecodeParams& p, int nt, int ctas, cudaStream_t stream);

// Device words that append and decode set: [0] on a bad page number or
// length, [1] on a wait that ran out of time; null where no call has set them
// up on this device.
int* page_error_words(int dev);

// of attn_host.cu: the launch counter, the bound on a wait, the test hook
void count_launch(int n);
unsigned long long wait_timeout_ns();
int skip_first_load();

}  // namespace attn
