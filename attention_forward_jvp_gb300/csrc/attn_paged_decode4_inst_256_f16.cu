// Decode over a cache in 4 bits, key head dim 256, queries and outputs in f16.
#include "attn_paged_decode4_kernel.cuh"

namespace attn {
template cudaError_t launch_decode4<256, 64, true>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<256, 128, true>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<256, 256, true>(Decode4Params&, int, int, cudaStream_t);
}  // namespace attn
