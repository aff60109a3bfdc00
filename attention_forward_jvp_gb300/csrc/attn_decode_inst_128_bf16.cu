// The paged decode kernels of key width 128, bf16 storage.
#include "attn_decode_tc_kernel.cuh"

namespace attn {
template cudaError_t launch_decode<128, 64, false>(DecodeParams&, int, int, cudaStream_t);
template cudaError_t launch_decode<128, 128, false>(DecodeParams&, int, int, cudaStream_t);
template cudaError_t launch_decode<128, 256, false>(DecodeParams&, int, int, cudaStream_t);
}  // namespace attn
