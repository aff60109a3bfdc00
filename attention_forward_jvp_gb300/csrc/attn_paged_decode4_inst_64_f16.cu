// Decode over a cache in 4 bits, key head dim 64, queries and outputs in f16.
#include "attn_paged_decode4_kernel.cuh"

namespace attn {
template cudaError_t launch_decode4<64, 64, true>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<64, 128, true>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<64, 256, true>(Decode4Params&, int, int, cudaStream_t);
}  // namespace attn
