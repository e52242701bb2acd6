#include "block_norm.cuh"

namespace moe {

cudaError_t block_norm_bf16(const BlockNormArgs& a, cudaStream_t s) { return fwd_t<__nv_bfloat16>(a, s); }

}  // namespace moe
