// The paged decode kernels of key width 256, bf16 storage.
#include "attn_decode_tc_kernel.cuh"

namespace attn {
template cudaError_t launch_decode<256, 64, false>(DecodeParams&, int, int, cudaStream_t);
template cudaError_t launch_decode<256, 128, false>(DecodeParams&, int, int, cudaStream_t);
template cudaError_t launch_decode<256, 256, false>(DecodeParams&, int, int, cudaStream_t);
}  // namespace attn
