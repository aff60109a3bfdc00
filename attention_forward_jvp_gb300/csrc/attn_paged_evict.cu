// Eviction (attn_paged_evict, attn_paged_evict4): of each key head of a
// sequence that is longer than it may stay, the tokens with the largest
// weights, the first and the last, copied in their order into fewer pages.
//
// Two kernels.  `select` has a block for each (sequence, key head): a radix
// selection of the M-th largest weight, in four passes of eight bits over
// weights turned to whole numbers of the same order, then the numbers of the
// kept tokens in order, each warp counting what a stretch of the row keeps
// before all write.  Ties go by the same order, so that the choice is a
// function of the weights alone.  `move` copies the rows of the kept tokens,
// 16 bytes a thread, several rows on their way.
//
// What bounds it: memory, the kept rows read and written once; the selection
// reads a head's weights six times, from L2 after the first.
#include "attn_paged_cache_kernels.h"
#include "ptx.cuh"

namespace attn {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;

// whole numbers in the order of the weights: -0 as 0, NaN above all
__device__ __forceinline__ uint32_t ordered(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// what a sequence has and keeps
struct Share {
  int n, keep, sinks, recent;
  bool over, odd;
};
__device__ __forceinline__ Share share_of(const EvictParams& p, int b) {
  Share s;
  s.n = p.seq_lens[b];
  s.odd = s.n < 0 || s.n > p.capacity;
  s.n = s.n < 0 ? 0 : min(s.n, p.capacity);
  s.keep = max(p.keep != nullptr ? p.keep[b] : p.keep_all, 0);
  s.over = s.n > s.keep;
  if (s.over && s.keep > p.new_capacity) {
    s.keep = p.new_capacity;
    s.odd = true;
  }
  s.recent = min(p.recent, s.keep);
  s.sinks = min(p.sinks, s.keep - s.recent);
  return s;
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int histogram[256];
  __shared__ int found[2];                      // the digit, the numbers above it
  __shared__ int counts[2][kSelectWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Share s = share_of(p, b);
  if (h == 0) {
    if (s.odd && tid == 0) *p.err = 1;
    if (tid == 0) p.lens_out[b] = min(s.n, s.keep);
    for (int i = tid; i < p.max_pages; i += kSelectThreads)
      p.table_out[b * p.table_out_stride + i] =
          s.over && i < p.n_new ? p.pages[b * p.pages_stride + i] : p.page_table[b * p.table_stride + i];
  }
  const float* w = p.w + b * p.ws[0] + h * p.ws[1];
  float* to = p.w_out + b * p.wos[0] + h * p.wos[1];
  if (!s.over) {
    for (long long i = tid; i < p.places; i += kSelectThreads) to[i] = w[i];
    return;
  }
  for (long long i = s.keep + tid; i < p.places; i += kSelectThreads) to[i] = 0.f;

  // the others' weights lie in [lo, hi); `most` of them are kept
  const int lo = s.sinks, hi = s.n - s.recent, most = s.keep - s.sinks - s.recent;
  uint32_t least = 0;  // the smallest kept number
  int ties = 0;        // how many that are equal to it
  if (most > 0) {
    int left = most;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) histogram[tid] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kSelectThreads) {
        const uint32_t u = ordered(w[i]);
        if (shift == 24 || u >> (shift + 8) == least) atomicAdd(&histogram[u >> shift & 255], 1);
      }
      __syncthreads();
      if (warp == 0) {  // the digits from the largest on, eight to a lane
        int c[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += c[j] = histogram[255 - 8 * lane - j];
        int above = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kAll, above, o);
          if (lane >= o) above += y;
        }
        above -= sum;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (above < left && above + c[j] >= left) {
            found[0] = 255 - 8 * lane - j;
            found[1] = above;
          }
          above += c[j];
        }
      }
      __syncthreads();
      least = least << 8 | static_cast<uint32_t>(found[0]);
      left -= found[1];
    }
    ties = left;
  }
  // each warp's stretch of the row: what it keeps for its weight, its ties
  const int each = ((s.n + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
  const int from = min(warp * each, s.n), end = min(from + each, s.n);
  int above = 0, equal = 0;
  for (int i = from; i < end; i += 32) {
    const int j = i + lane;
    const bool in = j < end, sure = in && (j < lo || j >= hi);
    const uint32_t u = in ? ordered(w[j]) : 0u;
    above += __popc(__ballot_sync(kAll, sure || (in && most > 0 && u > least)));
    equal += __popc(__ballot_sync(kAll, in && !sure && most > 0 && u == least));
  }
  if (lane == 0) {
    counts[0][warp] = above;
    counts[1][warp] = equal;
  }
  __syncthreads();
  int equals = lane < warp ? counts[1][lane] : 0, aboves = lane < warp ? counts[0][lane] : 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    equals += __shfl_xor_sync(kAll, equals, o);
    aboves += __shfl_xor_sync(kAll, aboves, o);
  }
  // places of the stretch: behind what the warps before it keep
  int at = aboves + min(equals, ties);
  int* index = p.index + static_cast<long long>(blockIdx.x) * p.new_capacity;
  for (int i = from; i < end; i += 32) {
    const int j = i + lane;
    const bool in = j < end, sure = in && (j < lo || j >= hi);
    const float x = in ? w[j] : 0.f;
    const uint32_t u = in ? ordered(x) : 0u;
    const bool tie = in && !sure && most > 0 && u == least;
    const unsigned all_ties = __ballot_sync(kAll, tie);
    const bool keep = sure || (in && most > 0 && u > least) ||
                      (tie && equals + __popc(all_ties & ((1u << lane) - 1)) < ties);
    const unsigned kept = __ballot_sync(kAll, keep);
    if (keep) {
      const int k = at + __popc(kept & ((1u << lane) - 1));
      index[k] = j;
      to[k] = x;
    }
    at += __popc(kept);
    equals += __popc(all_ties);
  }
}

constexpr int kMoveThreads = 256, kMoveUnroll = 4;

// Rows of keys (blockIdx.y 0) or values, 16 bytes a thread; the first thread of
// a row of 4 bits takes its steps and least values too.
template <int BITS>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictParams p, int chunks,
                                                            long long blocks) {
  constexpr int U = kMoveUnroll;
  griddep_wait();
  griddep_launch_dependents();
  const bool values = blockIdx.y != 0;
  const int d = values ? p.Dv : p.Dqk;
  const Pool4& pool = values ? p.v : p.k;
  const long long* st = BITS == 4 ? pool.st : (values ? p.vp : p.kp);
  char* base = BITS == 4 ? reinterpret_cast<char*>(pool.codes) : reinterpret_cast<char*>(values ? p.v16 : p.k16);
  const int items = d * BITS / 128;  // a power of two
  const int rows = kMoveThreads / items, item = threadIdx.x & (items - 1);
  constexpr int E = BITS == 4 ? 1 : 2;  // bytes of a unit of the strides
  for (long long x = blockIdx.x; x < blocks; x += gridDim.x) {
    const int bh = static_cast<int>(x / chunks), chunk = static_cast<int>(x - static_cast<long long>(bh) * chunks);
    const int b = bh / p.Hkv, h = bh - b * p.Hkv;
    const Share s = share_of(p, b);
    const long long first = static_cast<long long>(chunk) * rows * U;
    if (!s.over || first >= s.keep) continue;
    const int* index = p.index + static_cast<long long>(bh) * p.new_capacity;
    uint4 v[U], sc[U];
    long long to[U], to_scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long j = first + u * rows + threadIdx.x / items;
      to[u] = to_scale[u] = -1;
      v[u] = sc[u] = make_uint4(0u, 0u, 0u, 0u);
      if (j < s.keep) {
        const int i = index[j], k = static_cast<int>(j);
        const int src_e = i / p.page_size, dst_e = k / p.page_size;
        const int src_slot = i - src_e * p.page_size, dst_slot = k - dst_e * p.page_size;
        const int src = p.page_table[b * p.table_stride + src_e], dst = p.pages[b * p.pages_stride + dst_e];
        const bool from = static_cast<unsigned>(src) < static_cast<unsigned>(p.n_pages);
        const bool there = static_cast<unsigned>(dst) < static_cast<unsigned>(p.n_pages);
        if (!(from && there) && item == 0) *p.err = 1;
        if (there) to[u] = E * (dst * st[0] + h * st[1] + dst_slot * st[2]) + 16 * item;
        if (from) v[u] = *reinterpret_cast<const uint4*>(base + E * (src * st[0] + h * st[1] + src_slot * st[2]) + 16 * item);
        if (BITS == 4 && item == 0) {
          const uint16_t* a = pool.scales + src * pool.ss[0] + h * pool.ss[1] + src_slot * pool.ss[2];
          if (there) to_scale[u] = dst * pool.ss[0] + h * pool.ss[1] + dst_slot * pool.ss[2];
          if (from) {
            if (d <= 64) sc[u].x = *reinterpret_cast<const uint32_t*>(a);
            else if (d == 128) *reinterpret_cast<uint2*>(&sc[u]) = *reinterpret_cast<const uint2*>(a);
            else sc[u] = *reinterpret_cast<const uint4*>(a);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (to[u] >= 0) *reinterpret_cast<uint4*>(base + to[u]) = v[u];
      if (BITS == 4 && to_scale[u] >= 0) {
        uint16_t* a = pool.scales + to_scale[u];
        if (d <= 64) *reinterpret_cast<uint32_t*>(a) = sc[u].x;
        else if (d == 128) *reinterpret_cast<uint2*>(a) = make_uint2(sc[u].x, sc[u].y);
        else *reinterpret_cast<uint4*>(a) = sc[u];
      }
    }
  }
}

template <class K, class... A>
cudaError_t launch(K kernel, dim3 grid, int threads, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int bits, cudaStream_t stream, int* launches) {
  *launches = 1;
  cudaError_t e = launch(select_kernel, dim3(static_cast<unsigned>(p.B * p.Hkv)), kSelectThreads, stream, p);
  if (e != cudaSuccess || p.new_capacity == 0) return e;
  const int most = p.Dqk > p.Dv ? p.Dqk : p.Dv;
  const int fewest = kMoveThreads / (most * bits / 128) * kMoveUnroll;  // rows of a block, of the wider pool
  const int kept = p.keep == nullptr && p.keep_all < p.new_capacity ? (p.keep_all < 0 ? 0 : p.keep_all) : p.new_capacity;
  const int chunks = (kept + fewest - 1) / fewest;
  if (chunks == 0) return cudaSuccess;
  const long long blocks = static_cast<long long>(chunks) * p.B * p.Hkv;
  *launches = 2;
  const dim3 grid(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)), 2);
  return bits == 4 ? launch(move_kernel<4>, grid, kMoveThreads, stream, p, chunks, blocks)
                   : launch(move_kernel<16>, grid, kMoveThreads, stream, p, chunks, blocks);
}

}  // namespace attn
