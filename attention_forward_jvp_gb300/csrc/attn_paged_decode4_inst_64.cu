// Decode over a cache in 4 bits for the key head dim 64.
#include "attn_paged_decode4_kernel.cuh"

namespace attn {
template cudaError_t launch_decode4<64, 64>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<64, 128>(Decode4Params&, int, int, cudaStream_t);
template cudaError_t launch_decode4<64, 256>(Decode4Params&, int, int, cudaStream_t);
}  // namespace attn
