// Decode over a cache in 4 bits, key head dim 256, queries and outputs in bf16.
#include "attn_paged_decode4_kernel.cuh"

namespace attn {
template cudaError_t launch_decode4<256, 64, false>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<256, 128, false>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<256, 256, false>(Decode4Params&, int, int, cudaStream_t);
}  // namespace attn
