// Decode over a cache in 4 bits, key head dim 128, queries and outputs in f16.
#include "attn_paged_decode4_kernel.cuh"

namespace attn {
template cudaError_t launch_decode4<128, 64, true>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<128, 128, true>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<128, 256, true>(Decode4Params&, int, int, cudaStream_t);
}  // namespace attn
