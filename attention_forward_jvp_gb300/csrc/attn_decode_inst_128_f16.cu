// The paged decode kernels of key width 128, f16 storage.
#include "attn_decode_tc_kernel.cuh"

namespace attn {
template cudaError_t launch_decode<128, 64, true>(DecodeParams&, int, int, cudaStream_t);
template cudaError_t launch_decode<128, 128, true>(DecodeParams&, int, int, cudaStream_t);
template cudaError_t launch_decode<128, 256, true>(DecodeParams&, int, int, cudaStream_t);
}  // namespace attn
