// Host side of attn_paged.h: argument validation, frequencies, dispatch.
#include "attn_paged.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <mutex>

#include "attn_paged_host.h"
#include "attn_paged_kernels.h"

namespace attn {

#define ATTN_DECODE_DECL(DQ, DV)                                                                         \
  extern template cudaError_t launch_decode<DQ, DV, false>(DecodeParams&, int, int, cudaStream_t);       \
  extern template cudaError_t launch_decode<DQ, DV, true>(DecodeParams&, int, int, cudaStream_t);
ATTN_DECODE_DECL(64, 64)
ATTN_DECODE_DECL(64, 128)
ATTN_DECODE_DECL(64, 256)
ATTN_DECODE_DECL(128, 64)
ATTN_DECODE_DECL(128, 128)
ATTN_DECODE_DECL(128, 256)
ATTN_DECODE_DECL(256, 64)
ATTN_DECODE_DECL(256, 128)
ATTN_DECODE_DECL(256, 256)

namespace {

constexpr int kMaxDevices = 64;

// The words that append and decode set on a bad page number or length, and
// on a wait that ran out of time: fixed device variables, so that no call
// allocates.
__device__ int g_page_error[2];

std::mutex g_mu;
Device g_dev[kMaxDevices];

}  // namespace

attn_status device(Device* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ATTN_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  Device& d = g_dev[dev];
  if (d.err == nullptr) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return ATTN_ERR_CUDA;
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_page_error) != cudaSuccess || p == nullptr) return ATTN_ERR_CUDA;
    d.sms = sms;
    d.err = static_cast<int*>(p);
  }
  *out = d;
  return ATTN_OK;
}

namespace {

attn_status run_rope(int32_t B, int64_t N, int32_t D, const attn_rope_spec* rope, const attn_rope_tensor* tensors,
                     int32_t n_tensors, const int32_t* positions, const int64_t* pos_stride, const int32_t* offsets,
                     int32_t n_seq, int inverse, void* stream, bool f16) {
  if (rope == nullptr || tensors == nullptr || B < 0 || N < 0 || n_tensors < 1 || n_tensors > kRopeTensors)
    return ATTN_ERR_INVALID_ARG;
  if (D < 1 || D > 1024) return ATTN_ERR_UNSUPPORTED;
  if (N > 0x7fffffffLL || (offsets != nullptr && (B != 1 || n_seq < 0)) || (positions != nullptr && pos_stride == nullptr))
    return ATTN_ERR_INVALID_ARG;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  attn_status st = spec_of(rope, D, inverse != 0, &p.r);
  if (st != ATTN_OK) return st;
  bool vec = D % 16 == 0 && p.r.rot % 16 == 0;
  const bool rows = B > 0 && N > 0 && !(offsets != nullptr && n_seq == 0);
  for (int i = 0; i < n_tensors; ++i) {
    const attn_rope_tensor& t = tensors[i];
    if (t.H < 0) return ATTN_ERR_INVALID_ARG;
    if (t.H == 0 || !rows) continue;
    if (t.x == nullptr || t.y == nullptr) return ATTN_ERR_INVALID_ARG;
    if (!aligned(t.x, 2) || !aligned(t.y, 2)) return ATTN_ERR_MISALIGNED;
    RopeTensor& a = p.t[p.n_tensors++];
    a.x = static_cast<const uint16_t*>(t.x);
    a.y = static_cast<uint16_t*>(t.y);
    a.H = t.H;
    if (p.heads > 0x7fffffff - t.H) return ATTN_ERR_INVALID_ARG;
    p.heads += t.H;
    const int64_t sizes[3] = {B, t.H, N};
    const bool xs8 = take_strides(t.x_stride, sizes, 3, a.xs), ys8 = take_strides(t.y_stride, sizes, 3, a.ys);
    if (t.x == t.y && std::memcmp(a.xs, a.ys, sizeof(a.xs)) != 0) return ATTN_ERR_INVALID_ARG;
    if (shares_places(sizes, 3, a.ys)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j + 1 < p.n_tensors; ++j)
      if (a.y == p.t[j].y || a.y == p.t[j].x || a.x == p.t[j].y) return ATTN_ERR_INVALID_ARG;
    vec = vec && xs8 && ys8 && aligned16(t.x) && aligned16(t.y);
  }
  if (p.heads == 0) return ATTN_OK;
  if (positions != nullptr && !aligned(positions, 4)) return ATTN_ERR_MISALIGNED;
  if (offsets != nullptr && !aligned(offsets, 4)) return ATTN_ERR_MISALIGNED;
  Device d;
  st = device(&d);
  if (st != ATTN_OK) return st;
  p.D = D;
  p.N = N;
  p.rows = static_cast<long long>(B) * N;
  p.positions = positions;
  if (positions != nullptr) {
    p.ps[0] = pos_stride[0];
    p.ps[1] = pos_stride[1];
  }
  p.offsets = offsets;
  p.n_seq = n_seq;
  const int items = vec ? D / 16 : D - p.r.rot / 2;
  const int splits = head_splits(p.rows * items, p.heads, d.sms, &p.heads_per_split);
  if (launch_rope(p, vec, f16, splits, static_cast<cudaStream_t>(stream)) != cudaSuccess) return ATTN_ERR_CUDA;
  count_launch(1);
  return ATTN_OK;
}

attn_status run_append(const attn_paged_cache* c, const attn_paged_new* n, const attn_rope_spec* rope, void* stream,
                       bool f16) {
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  attn_status st = check_cache(c, p.kp, p.vp);
  if (st != ATTN_OK) return st;
  if (n == nullptr || n->T < 0 || n->T > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  if (n->offsets == nullptr && n->T != c->B) return ATTN_ERR_INVALID_ARG;
  if (n->q != nullptr && (n->Hq < 0 || n->q_out == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (rope != nullptr) {
    st = spec_of(rope, c->Dqk, false, &p.r);
    if (st != ATTN_OK) return st;
  }
  if (c->B == 0 || n->T == 0) return ATTN_OK;
  if (n->k == nullptr || n->v == nullptr) return ATTN_ERR_INVALID_ARG;
  for (const void* x : {n->k, n->v, n->q, static_cast<const void*>(n->q_out)})
    if (!aligned(x, 2)) return ATTN_ERR_MISALIGNED;
  if (!aligned(n->offsets, 4)) return ATTN_ERR_MISALIGNED;
  const int64_t kv_sizes[2] = {n->T, c->Hkv}, q_sizes[2] = {n->T, n->Hq};
  const bool k8 = take_strides(n->k_stride, kv_sizes, 2, p.ks), v8 = take_strides(n->v_stride, kv_sizes, 2, p.vs);
  bool vec = p.r.rot % 16 == 0 && k8 && v8 && aligned16(n->k) && aligned16(n->v);
  if (n->q != nullptr) {
    const bool q8 = take_strides(n->q_stride, q_sizes, 2, p.qs), o8 = take_strides(n->q_out_stride, q_sizes, 2, p.qos);
    if (n->q == n->q_out && std::memcmp(p.qs, p.qos, sizeof(p.qs)) != 0) return ATTN_ERR_INVALID_ARG;
    if (shares_places(q_sizes, 2, p.qos)) return ATTN_ERR_INVALID_ARG;
    if (n->Hq > 0 && (n->q_out == n->k || n->q_out == n->v)) return ATTN_ERR_INVALID_ARG;
    vec = vec && q8 && o8 && aligned16(n->q) && aligned16(n->q_out);
  }
  const int64_t pool_sizes[3] = {c->n_pages, c->Hkv, c->page_size};
  if (shares_places(pool_sizes, 3, p.kp) || shares_places(pool_sizes, 3, p.vp)) return ATTN_ERR_INVALID_ARG;
  // one pool for both holds what both write only where that is the same
  if (c->n_pages > 0 && c->k == c->v && (rope != nullptr || n->k != n->v)) return ATTN_ERR_INVALID_ARG;
  Device d;
  st = device(&d);
  if (st != ATTN_OK) return st;
  p.k = static_cast<const uint16_t*>(n->k);
  p.v = static_cast<const uint16_t*>(n->v);
  p.q = static_cast<const uint16_t*>(n->q);
  p.q_out = static_cast<uint16_t*>(n->q_out);
  p.k_pool = static_cast<uint16_t*>(c->k);
  p.v_pool = static_cast<uint16_t*>(c->v);
  p.Hq = n->q != nullptr ? n->Hq : 0;
  p.Hkv = c->Hkv;
  p.Dqk = c->Dqk;
  p.Dv = c->Dv;
  p.T = n->T;
  p.offsets = n->offsets;
  p.page_table = c->page_table;
  p.table_stride = c->table_stride;
  p.seq_lens = c->seq_lens;
  p.B = c->B;
  p.max_pages = c->max_pages;
  p.n_pages = c->n_pages;
  p.page_size = c->page_size;
  p.err = d.err;
  const int64_t heads = static_cast<int64_t>(p.Hq) + 2 * static_cast<int64_t>(p.Hkv);
  if (heads > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  const int qk = vec ? p.Dqk / 16 : p.Dqk - p.r.rot / 2, v = vec ? p.Dv / 16 : p.Dv;
  const int splits = head_splits(p.T * (qk > v ? qk : v), static_cast<int>(heads), d.sms, &p.heads_per_split);
  if (launch_append(p, vec, f16, splits, static_cast<cudaStream_t>(stream)) != cudaSuccess) return ATTN_ERR_CUDA;
  count_launch(1);
  return ATTN_OK;
}

// ------------------------------------------------------------------- decode
// How the kernel runs a cache's head dims and Hq query heads
struct Layout {
  int dq, dv;          // kernel head dims
  int rows, chunks;    // query heads of a unit, units of a key head
  int nt;              // groups of 8 query heads; 0: more than the warps' kernel takes
  int ctas;
  size_t desc, ml, total;  // workspace: bytes of the first two parts, of all
};
Layout layout_of(const attn_paged_cache* c, int Hq, int sms) {
  Layout l;
  l.dq = c->Dqk < 64 ? 64 : c->Dqk;
  l.dv = c->Dv < 64 ? 64 : c->Dv;
  const int G = Hq / c->Hkv;
  l.chunks = (G + kDecodeMaxRows - 1) / kDecodeMaxRows;
  l.rows = (G + l.chunks - 1) / l.chunks;
  l.nt = l.rows > decode_warp_rows(l.dq, l.dv) ? 0 : (l.rows + 7) / 8;
  l.ctas = sms;
  const size_t warps = static_cast<size_t>(sms) * (l.nt == 0 ? 1 : kDecodeMaxWarps);  // ranges
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l.desc = up(sizeof(int4) * warps);
  l.ml = up(sizeof(float2) * 2 * warps * l.rows);
  l.total = l.desc + l.ml + sizeof(float) * 2 * warps * static_cast<size_t>(l.rows) * l.dv;
  return l;
}

template <bool F16>
cudaError_t dispatch_decode(const Layout& l, DecodeParams& p, cudaStream_t s) {
  switch (l.dq * 1000 + l.dv) {
    case 64064: return launch_decode<64, 64, F16>(p, l.nt, l.ctas, s);
    case 64128: return launch_decode<64, 128, F16>(p, l.nt, l.ctas, s);
    case 64256: return launch_decode<64, 256, F16>(p, l.nt, l.ctas, s);
    case 128064: return launch_decode<128, 64, F16>(p, l.nt, l.ctas, s);
    case 128128: return launch_decode<128, 128, F16>(p, l.nt, l.ctas, s);
    case 128256: return launch_decode<128, 256, F16>(p, l.nt, l.ctas, s);
    case 256064: return launch_decode<256, 64, F16>(p, l.nt, l.ctas, s);
    case 256128: return launch_decode<256, 128, F16>(p, l.nt, l.ctas, s);
    case 256256: return launch_decode<256, 256, F16>(p, l.nt, l.ctas, s);
  }
  return cudaErrorInvalidValue;
}

attn_status check_heads(const attn_paged_cache* c, int Hq) {
  return Hq >= 0 && Hq % c->Hkv == 0 ? ATTN_OK : ATTN_ERR_INVALID_ARG;
}

attn_status run_decode(const attn_paged_cache* c, int32_t Hq, const void* q, const int64_t* q_stride, float sm_scale,
                       void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream, bool f16) {
  DecodeParams p;
  std::memset(&p, 0, sizeof(p));
  attn_status st = check_cache(c, p.kp, p.vp);
  if (st == ATTN_OK) st = check_heads(c, Hq);
  if (st != ATTN_OK) return st;
  if (!std::isnan(sm_scale) && !(sm_scale > 0.f && std::isfinite(sm_scale))) return ATTN_ERR_INVALID_ARG;
  if (c->B == 0 || Hq == 0) return ATTN_OK;
  if (q == nullptr || q_stride == nullptr || o == nullptr || lse == nullptr || workspace == nullptr)
    return ATTN_ERR_INVALID_ARG;
  const int64_t q_sizes[2] = {c->B, Hq};
  if (!take_strides(q_stride, q_sizes, 2, p.qs) || !aligned16(q) || !aligned16(o) || !aligned(lse, 4) ||
      !aligned16(workspace))
    return ATTN_ERR_MISALIGNED;
  Device d;
  st = device(&d);
  if (st != ATTN_OK) return st;
  const Layout l = layout_of(c, Hq, d.sms);
  if (workspace_bytes < l.total) return ATTN_ERR_INVALID_ARG;
  if (static_cast<int64_t>(c->Hkv) * l.chunks > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(c->k);
  p.v = static_cast<const uint16_t*>(c->v);
  p.page_table = c->page_table;
  p.table_stride = c->table_stride;
  p.seq_lens = c->seq_lens;
  p.B = c->B;
  p.n_pages = c->n_pages;
  p.page_size = c->page_size;
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (c->page_size == 1 << s) p.page_shift = s;
  const int64_t cap = static_cast<int64_t>(c->max_pages) * c->page_size;
  p.capacity = static_cast<int>(cap < (1 << 30) ? cap : (1 << 30));
  p.Hkv = c->Hkv;
  p.G = Hq / c->Hkv;
  p.rows = l.rows;
  p.chunks = l.chunks;
  p.dqk = c->Dqk;
  p.dv = c->Dv;
  p.whole = c->page_size % kDecodeBN == 0 ? 1 : 0;
  const float scale = std::isnan(sm_scale) ? 1.0f / std::sqrt(static_cast<float>(c->Dqk)) : sm_scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  p.desc = reinterpret_cast<int4*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + l.desc);
  p.part_o = reinterpret_cast<float*>(ws + l.desc + l.ml);
  p.err = d.err;
  p.timeout_ns = wait_timeout_ns();
  p.skip_first_load = skip_first_load();
  p.split = p.capacity > kDecodeBN ? 1 : 0;
  const double steps = (p.capacity / kDecodeBN + 1.0) * p.B * p.Hkv * p.chunks;
  p.wide = steps + l.ctas * kDecodeMaxWarps < 2147483648.0 ? 0 : 1;
  const cudaError_t e = f16 ? dispatch_decode<true>(l, p, static_cast<cudaStream_t>(stream))
                            : dispatch_decode<false>(l, p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  count_launch(1 + p.split);
  return ATTN_OK;
}

}  // namespace

int* page_error_words(int dev) {
  std::lock_guard<std::mutex> lk(g_mu);
  return dev >= 0 && dev < kMaxDevices ? g_dev[dev].err : nullptr;
}

}  // namespace attn

extern "C" {

attn_status attn_rope(int32_t B, int64_t N, int32_t D, const attn_rope_spec* rope, const attn_rope_tensor* tensors,
                      int32_t n_tensors, const int32_t* positions, const int64_t pos_stride[2],
                      const int32_t* offsets, int32_t n_seq, int inverse, void* stream) {
  return attn::run_rope(B, N, D, rope, tensors, n_tensors, positions, pos_stride, offsets, n_seq, inverse, stream,
                        false);
}
attn_status attn_rope_f16(int32_t B, int64_t N, int32_t D, const attn_rope_spec* rope,
                          const attn_rope_tensor* tensors, int32_t n_tensors, const int32_t* positions,
                          const int64_t pos_stride[2], const int32_t* offsets, int32_t n_seq, int inverse,
                          void* stream) {
  return attn::run_rope(B, N, D, rope, tensors, n_tensors, positions, pos_stride, offsets, n_seq, inverse, stream,
                        true);
}

attn_status attn_rope_freqs(const attn_rope_freq* f, double* inv_freq) {
  if (f == nullptr || inv_freq == nullptr) return ATTN_ERR_INVALID_ARG;
  if (f->rot_dim <= 0 || f->rot_dim % 2 != 0) return ATTN_ERR_INVALID_ARG;
  if (!(f->base > 0) || !std::isfinite(f->base)) return ATTN_ERR_INVALID_ARG;
  const int kind = f->scaling;
  if (kind < ATTN_ROPE_SCALE_NONE || kind > ATTN_ROPE_SCALE_BY_PARTS) return ATTN_ERR_INVALID_ARG;
  if (kind != ATTN_ROPE_SCALE_NONE && (!(f->factor > 0) || !std::isfinite(f->factor))) return ATTN_ERR_INVALID_ARG;
  double base = f->base;
  if (kind == ATTN_ROPE_SCALE_BASE) {
    if (f->rot_dim == 2) return ATTN_ERR_INVALID_ARG;  // one frequency, the highest: the base has no say
    base *= std::pow(f->factor, static_cast<double>(f->rot_dim) / (f->rot_dim - 2));
    if (!(base > 0) || !std::isfinite(base)) return ATTN_ERR_INVALID_ARG;
  }
  if (kind == ATTN_ROPE_SCALE_BY_PARTS &&
      (!(f->orig_len > 0) || !std::isfinite(f->orig_len) || !(f->low_turns >= 0) ||
       !(f->high_turns > f->low_turns) || !std::isfinite(f->high_turns)))
    return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < f->rot_dim / 2; ++i) {
    double w = std::pow(base, -2.0 * i / f->rot_dim);
    if (kind == ATTN_ROPE_SCALE_LINEAR) w /= f->factor;
    if (kind == ATTN_ROPE_SCALE_BY_PARTS) {
      const double turns = f->orig_len * w / 6.283185307179586476925;
      double keep = (turns - f->low_turns) / (f->high_turns - f->low_turns);
      keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
      w = w * keep + w / f->factor * (1 - keep);
    }
    if (!std::isfinite(w)) return ATTN_ERR_INVALID_ARG;
    inv_freq[i] = w;
  }
  return ATTN_OK;
}

attn_status attn_rope_steps(const double* inv_freq, int32_t n, uint64_t* steps) {
  if (n < 0 || (n > 0 && (inv_freq == nullptr || steps == nullptr))) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i])) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    double turn = inv_freq[i] / 6.283185307179586476925;
    turn -= std::floor(turn);
    // (a turn that the subtraction rounded to 1 is a full one: no step)
    const double x = std::ldexp(turn, 64);
    steps[i] = x >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(x);
  }
  return ATTN_OK;
}

attn_status attn_paged_append(const attn_paged_cache* cache, const attn_paged_new* tokens, const attn_rope_spec* rope,
                              void* stream) {
  return attn::run_append(cache, tokens, rope, stream, false);
}
attn_status attn_paged_append_f16(const attn_paged_cache* cache, const attn_paged_new* tokens,
                                  const attn_rope_spec* rope, void* stream) {
  return attn::run_append(cache, tokens, rope, stream, true);
}

size_t attn_paged_decode_workspace(const attn_paged_cache* cache, int32_t Hq) {
  long long kp[3], vp[3];
  if (attn::check_cache(cache, kp, vp) != ATTN_OK || attn::check_heads(cache, Hq) != ATTN_OK || cache->B == 0 ||
      Hq == 0)
    return 0;
  attn::Device d;
  if (attn::device(&d) != ATTN_OK) return 0;
  return attn::layout_of(cache, Hq, d.sms).total;
}
attn_status attn_paged_decode(const attn_paged_cache* cache, int32_t Hq, const void* q, const int64_t q_stride[2],
                              float sm_scale, void* o, float* lse, void* workspace, size_t workspace_bytes,
                              void* stream) {
  return attn::run_decode(cache, Hq, q, q_stride, sm_scale, o, lse, workspace, workspace_bytes, stream, false);
}
attn_status attn_paged_decode_f16(const attn_paged_cache* cache, int32_t Hq, const void* q,
                                  const int64_t q_stride[2], float sm_scale, void* o, float* lse, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return attn::run_decode(cache, Hq, q, q_stride, sm_scale, o, lse, workspace, workspace_bytes, stream, true);
}

}  // extern "C"
