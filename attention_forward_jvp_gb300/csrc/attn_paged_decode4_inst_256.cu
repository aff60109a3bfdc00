// Decode over a cache in 4 bits for the key head dim 256.
#include "attn_paged_decode4_kernel.cuh"

namespace attn {
template cudaError_t launch_decode4<256, 64>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<256, 128>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<256, 256>(Decode4Params&, int, int, cudaStream_t);
}  // namespace attn
