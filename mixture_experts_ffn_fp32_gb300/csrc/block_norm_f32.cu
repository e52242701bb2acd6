#include "block_norm.cuh"

namespace moe {

cudaError_t block_norm_f32(const BlockNormArgs& a, cudaStream_t s) { return fwd_t<float>(a, s); }

}  // namespace moe
