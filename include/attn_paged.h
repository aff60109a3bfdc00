/*
 * attn_paged.h -- rotary positions, and the paged key-value cache with the
 * attention of one new token that reads it.  Part of the library of
 * attn_jvp.h: its status codes, stream and ownership conventions hold here.
 *
 *   attn_rope          rotates up to four tensors (q, k, their tangents, or
 *                      the gradients dq, dk with `inverse`) in one launch
 *   attn_paged_append  writes the keys and values of new tokens into the
 *                      pages of their sequences, rotating the keys (and the
 *                      queries, beside them) to their positions on the way
 *   attn_paged_decode  softmax attention of one query token per sequence
 *                      over its pages, split over the length and joined
 *
 * Types: bf16 storage; the *_f16 entry points take fp16.  Every product,
 * sum, angle and softmax statistic is fp32 or wider.
 *
 * Calls are asynchronous on `stream`, which belongs to the current device,
 * allocate no device memory, and may be captured into a graph.  Argument
 * errors are returned synchronously and launch nothing.  What only the
 * device can see (a page number or a length out of range) is refused there:
 * nothing outside the pool is read or written, and the next attn_sync_check
 * on the device returns ATTN_ERR_PAGE.
 *
 * Each kernel waits for the work before it on the stream, however it was
 * launched; calls on different streams share nothing but that error word.
 */
#ifndef ATTN_PAGED_H
#define ATTN_PAGED_H

#include <stddef.h>
#include <stdint.h>

#include "attn_jvp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------ rotary positions
 *
 * A head of D elements has its first rot_dim elements rotated in pairs:
 * pair i of position p turns by the angle p * inv_freq[i],
 *
 *   y_a = out_scale (x_a cos - x_b sin)
 *   y_b = out_scale (x_a sin + x_b cos)
 *
 * with (a, b) = (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved; the
 * other elements are copied.  `inverse` turns by the negative angle, which
 * (out_scale included) is the transpose: it takes the gradient of y to the
 * gradient of x.  The map is linear, so a tangent of x is rotated like x.
 *
 * `steps` is a DEVICE array of rot_dim / 2 words: the turn of pair i per
 * position as a fraction of a full turn, times 2^64, modulo 2^64
 * (attn_rope_steps).  position * step in 64-bit integers is then the angle
 * modulo a full turn, exactly, so far positions lose nothing. */
typedef struct {
  const uint64_t* steps;
  int32_t rot_dim;      /* even, 0 < rot_dim <= D */
  int32_t interleaved;
  float out_scale;      /* finite; 1 for the plain rotation */
} attn_rope_spec;

/* One tensor: x is read and y written, both [batch, head, token, D] by
 * strides (batch, head, token) in elements, the D elements of a row
 * contiguous.  y == x with equal strides rotates in place; any other
 * overlap is undefined, and refused where it shows: a y that is also another
 * tensor's x or y, a y stride of 0 over more than one element.  Rows that are 16-byte aligned (pointer and strides), with D and
 * rot_dim multiples of 16, move in 16-byte accesses; others element by
 * element. */
typedef struct {
  const void* x;
  void* y;
  int32_t H;
  int64_t x_stride[3];
  int64_t y_stride[3];
} attn_rope_tensor;

/* Rotates n_tensors (1 to 4) tensors of B x N tokens and D elements a head
 * (1 <= D <= 1024).
 *   positions  device int32, element (b, n) at b * pos_stride[0] +
 *              n * pos_stride[1] (a stride of 0 broadcasts); NULL: n, or the
 *              token's place in its sequence when jagged
 *   offsets    NULL, or the jagged layout of attn_fwd (B must be 1, N = T):
 *              device int32 [n_seq + 1], offsets[0] = 0, non-decreasing;
 *              rows >= offsets[n_seq] are not written
 * pos_stride is only read with positions, n_seq only with offsets. */
attn_status attn_rope(int32_t B, int64_t N, int32_t D, const attn_rope_spec* rope,
                      const attn_rope_tensor* tensors, int32_t n_tensors,
                      const int32_t* positions, const int64_t pos_stride[2],
                      const int32_t* offsets, int32_t n_seq, int inverse, void* stream);
attn_status attn_rope_f16(int32_t B, int64_t N, int32_t D, const attn_rope_spec* rope,
                          const attn_rope_tensor* tensors, int32_t n_tensors,
                          const int32_t* positions, const int64_t pos_stride[2],
                          const int32_t* offsets, int32_t n_seq, int inverse, void* stream);

/* How the frequencies inv_freq[i] = base^(-2 i / rot_dim) are stretched for
 * contexts longer than those trained on:
 *   NONE      as they are
 *   LINEAR    all divided by `factor` (positions interpolated)
 *   BASE      the base multiplied by factor^(rot_dim / (rot_dim - 2)), which
 *             divides the lowest frequency by `factor` and keeps the highest
 *   BY_PARTS  by the turns r = orig_len * inv_freq / (2 pi) that a pair makes
 *             over the trained context: divided by `factor` below low_turns,
 *             kept above high_turns, blended linearly in r between */
enum {
  ATTN_ROPE_SCALE_NONE = 0,
  ATTN_ROPE_SCALE_LINEAR = 1,
  ATTN_ROPE_SCALE_BASE = 2,
  ATTN_ROPE_SCALE_BY_PARTS = 3
};
typedef struct {
  int32_t rot_dim;
  int32_t scaling;     /* one of ATTN_ROPE_SCALE_* */
  double base;         /* > 0 */
  double factor;       /* > 0; not read for NONE */
  double orig_len;     /* BY_PARTS: > 0 */
  double low_turns;    /* BY_PARTS: >= 0 */
  double high_turns;   /* BY_PARTS: > low_turns */
} attn_rope_freq;

/* HOST functions, no GPU involved: the frequencies of a scaling
 * (inv_freq[rot_dim / 2], radians per position), and the steps of any n
 * frequencies (finite). */
attn_status attn_rope_freqs(const attn_rope_freq* freq, double* inv_freq);
attn_status attn_rope_steps(const double* inv_freq, int32_t n, uint64_t* steps);

/* ----------------------------------------------------------- paged cache
 *
 * Keys and values live in pools of pages of page_size tokens, each an array
 * [page, head, token in page, D] by strides (page, head, token) in elements,
 * the D elements of a row contiguous; pools that are token-major are the
 * same array by other strides.  Position p of sequence b is token
 * p % page_size of page page_table[b * table_stride + p / page_size].
 * seq_lens[b] is the number of tokens that sequence b holds, those of an
 * append in the same step included; 0 marks an idle place of the batch.
 *
 * Dqk, Dv each in {16, 32, 64, 128, 256}, independently; pools 16-byte
 * aligned with strides that are multiples of 8 elements
 * (ATTN_ERR_MISALIGNED).  Pool offsets are 64 bits wide. */
typedef struct {
  int32_t B;            /* sequences (places of the batch) */
  int32_t max_pages;    /* entries of a row of page_table */
  int32_t n_pages;      /* pages of the pool */
  int32_t page_size;
  int32_t Hkv, Dqk, Dv;
  void* k;
  void* v;
  int64_t k_stride[3];
  int64_t v_stride[3];
  const int32_t* page_table;  /* device [B, max_pages] */
  int64_t table_stride;       /* elements from row to row */
  const int32_t* seq_lens;    /* device [B] */
} attn_paged_cache;

/* New tokens, packed: k [T, Hkv, Dqk], v [T, Hkv, Dv] and, unless q is NULL,
 * q [T, Hq, Dqk] -> q_out, by strides (token, head) in elements, rows
 * contiguous.  offsets NULL: T = B, token b is the last of sequence b.
 * Else device int32 [B + 1] as in attn_rope: sequence b brings the
 * n_b = offsets[b + 1] - offsets[b] last of its seq_lens[b] tokens; rows
 * >= offsets[B] are left as they were. */
typedef struct {
  int64_t T;
  const int32_t* offsets;
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  int32_t Hq;
  int64_t k_stride[2];
  int64_t v_stride[2];
  int64_t q_stride[2];
  int64_t q_out_stride[2];
} attn_paged_new;

/* Writes each new token's key (rotated to its position, unless rope is
 * NULL) and value into its page, and its rotated query into q_out (q_out ==
 * q with equal strides: in place).  A token's position is seq_lens[b] - n_b
 * + its index.  An idle place's token (seq_lens[b] == 0, offsets NULL) and
 * one without a position (more tokens than seq_lens[b]) write nothing to
 * the cache and zeros to q_out; the latter, and a token whose position lies
 * behind the table's row or whose page is not in [0, n_pages), is reported
 * as ATTN_ERR_PAGE.  No two tokens of one call may share a place in the
 * pool; pools or a q_out with a stride of 0 over more than one element, one
 * pool for keys and values (a decode may read such pools) unless k is v and
 * nothing is rotated, and a q_out that is k or v are refused. */
attn_status attn_paged_append(const attn_paged_cache* cache, const attn_paged_new* tokens,
                              const attn_rope_spec* rope, void* stream);
attn_status attn_paged_append_f16(const attn_paged_cache* cache, const attn_paged_new* tokens,
                                  const attn_rope_spec* rope, void* stream);

/* For every sequence b and query head h (key head h / (Hq / Hkv); Hkv
 * divides Hq), over the keys j < seq_lens[b]:
 *
 *   S = sm_scale q K^T     O = softmax(S) V     LSE = log sum_j exp(S_j)
 *
 *   q   [B, Hq, Dqk] by strides (sequence, head), 16-byte aligned rows
 *   o   [B, Hq, Dv] contiguous, 16-byte aligned    lse [B, Hq] fp32
 *
 * sm_scale: NaN selects Dqk^-1/2, else positive and finite.  An idle place
 * gets O = 0 and LSE = -inf; its q is not read.  Whatever a page holds
 * behind a sequence's last token is never used.  A NaN among a head's keys
 * and values gives NaN, an infinite value infinity or NaN (probabilities are
 * multiplied in two parts, one of which may be 0 or negative); scores of
 * -inf have no weight, and a head with no others gets 0 and -inf.  A length outside [0, max_pages * page_size]
 * (2^30 at most) counts as the nearer bound, and a page not in [0, n_pages)
 * as keys and values of zero; both are reported as ATTN_ERR_PAGE.
 *
 * workspace: 16-byte aligned device memory of attn_paged_decode_workspace()
 * bytes (from the same cache and Hq, on the current device; 0 on an error)
 * for the parts of sequences that are split, written and read within the
 * call: its contents need not be kept or cleared, and calls that may overlap
 * on the GPU need one each.  Results do not depend on timing: the split is
 * a function of seq_lens and the shape, and parts are joined in order. */
size_t attn_paged_decode_workspace(const attn_paged_cache* cache, int32_t Hq);
attn_status attn_paged_decode(const attn_paged_cache* cache, int32_t Hq, const void* q, const int64_t q_stride[2],
                              float sm_scale, void* o, float* lse, void* workspace, size_t workspace_bytes,
                              void* stream);
attn_status attn_paged_decode_f16(const attn_paged_cache* cache, int32_t Hq, const void* q,
                                  const int64_t q_stride[2], float sm_scale, void* o, float* lse,
                                  void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_PAGED_H */
