// The norms on both sides of a block (block_norm.cuh): what their types share. The
// kernels of a type are compiled by a unit of its own.
#include "block_norm.cuh"

namespace moe {
namespace {

// The parameters' gradients from n partial rows, each column's sums in a fixed
// order: 32 threads take every 32nd row, then theirs are added in order.
constexpr int COL_ROWS = 32;
template <int NS>
__global__ void __launch_bounds__(32 * COL_ROWS)
block_norm_params_kernel(const __grid_constant__ BlockNormArgs a, int n, const float* __restrict__ part) {
    __shared__ float s[COL_ROWS][32];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    pdl_wait();
    pdl_trigger();
    float sum[NS];
#pragma unroll
    for (int q = 0; q < NS; ++q) {
        float v = 0.0f;
        if (c < a.d) {
            for (int r0 = ry; r0 < n; r0 += 10 * COL_ROWS) {
                float e[10];
#pragma unroll
                for (int i = 0; i < 10; ++i) {
                    const int r = r0 + i * COL_ROWS;
                    e[i] = r < n ? part[(static_cast<long long>(r) * NS + q) * a.d + c] : 0.0f;
                }
                v += (((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]))) + (e[8] + e[9]);
            }
        }
        s[ry][cx] = v;
        __syncthreads();
        v = s[0][cx];
#pragma unroll
        for (int i = 1; i < COL_ROWS; ++i) v += s[i][cx];
        sum[q] = v;
        __syncthreads();
    }
    if (ry != 0 || c >= a.d) return;
    const float s1 = sum[0], s2 = NS == 4 ? sum[NS / 2 - 1] : 0.0f, s3 = sum[NS / 2], s4 = NS == 4 ? sum[NS - 1] : 0.0f;
    const float g = weight(a.gate, c);
    if (a.dw != nullptr) a.dw[c] = s3;
    if (a.db != nullptr) a.db[c] = s4;
    if (a.dpost_w != nullptr) a.dpost_w[c] = g * s1;
    if (a.dpost_b != nullptr) a.dpost_b[c] = g * s2;
    if (a.dgate != nullptr) a.dgate[c] = a.post ? weight(a.post_w, c) * s1 + offset(a.post_b, c) * s2 : s1;
}

}  // namespace

cudaError_t launch_block_norm_params(const BlockNormArgs& a, int n, const float* part, cudaStream_t s) {
    const dim3 grid((a.d + 31) / 32), block(32 * COL_ROWS);
    return a.layer ? launch_pdl(block_norm_params_kernel<4>, grid, block, 0, s, a, n, part)
                   : launch_pdl(block_norm_params_kernel<2>, grid, block, 0, s, a, n, part);
}

size_t block_norm_bwd_floats(int R, int d, bool layer) {
    return static_cast<size_t>(bwd_parts(R, d)) * (layer ? 4 : 2) * d + (d > BWD_MAX_D ? 2 * static_cast<size_t>(R) : 0);
}

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s) {
    switch (a.dtype) {
        case MOE_BF16: return block_norm_bf16(a, s);
        case MOE_F16: return block_norm_f16(a, s);
        default: return block_norm_f32(a, s);
    }
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, float* ws, cudaStream_t s) {
    switch (a.dtype) {
        case MOE_BF16: return block_norm_bwd_bf16(a, ws, s);
        case MOE_F16: return block_norm_bwd_f16(a, ws, s);
        default: return block_norm_bwd_f32(a, ws, s);
    }
}

}  // namespace moe
