#include "block_norm.cuh"

namespace moe {

cudaError_t block_norm_bwd_f32(const BlockNormArgs& a, float* ws, cudaStream_t s) { return bwd_t<float>(a, ws, s); }

}  // namespace moe
