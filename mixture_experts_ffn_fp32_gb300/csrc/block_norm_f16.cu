#include "block_norm.cuh"

namespace moe {

cudaError_t block_norm_f16(const BlockNormArgs& a, cudaStream_t s) { return fwd_t<__half>(a, s); }

}  // namespace moe
