#include "block_norm.cuh"

namespace moe {

cudaError_t block_norm_bwd_bf16(const BlockNormArgs& a, float* ws, cudaStream_t s) { return bwd_t<__nv_bfloat16>(a, ws, s); }

}  // namespace moe
