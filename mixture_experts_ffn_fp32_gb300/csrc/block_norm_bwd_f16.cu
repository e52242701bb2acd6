#include "block_norm.cuh"

namespace moe {

cudaError_t block_norm_bwd_f16(const BlockNormArgs& a, float* ws, cudaStream_t s) { return bwd_t<__half>(a, ws, s); }

}  // namespace moe
