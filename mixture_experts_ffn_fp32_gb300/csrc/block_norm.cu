// The norms on both sides of a block (block_norm.cuh): what their types share. The
// kernels of a type are compiled by a unit of its own.
#include <algorithm>

#include "block_norm.cuh"

namespace moe {
namespace {

// The parameters' gradients from n partial rows, each column's sums in a fixed order:
// a CTA takes 8 columns (a sector of a row), 32 threads of each every 32nd row, and theirs
// are added in order.
constexpr int COLS = 8, SLOTS = 32;
template <int NS>
__global__ void __launch_bounds__(COLS * SLOTS)
block_norm_params_kernel(const __grid_constant__ BlockNormArgs a, int n, const float* __restrict__ part) {
    __shared__ float s[NS][SLOTS][COLS];
    const int cx = threadIdx.x % COLS, slot = threadIdx.x / COLS;
    const int c = blockIdx.x * COLS + cx;
    pdl_wait();
    pdl_trigger();
    float v[NS] = {};
    if (c < a.d) {
        for (int r0 = slot; r0 < n; r0 += 8 * SLOTS) {
            float e[8][NS];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = r0 + i * SLOTS;
#pragma unroll
                for (int q = 0; q < NS; ++q) e[i][q] = r < n ? part[(static_cast<long long>(r) * NS + q) * a.d + c] : 0.0f;
            }
#pragma unroll
            for (int q = 0; q < NS; ++q)
                v[q] += ((e[0][q] + e[1][q]) + (e[2][q] + e[3][q])) + ((e[4][q] + e[5][q]) + (e[6][q] + e[7][q]));
        }
    }
#pragma unroll
    for (int q = 0; q < NS; ++q) s[q][slot][cx] = v[q];
    __syncthreads();
    if (slot >= NS) return;
    float sum = s[slot][0][cx];
#pragma unroll
    for (int i = 1; i < SLOTS; ++i) sum += s[slot][i][cx];
    // the first warp: slot q has the columns' S(q + 1) (RMS: S1, S3)
    constexpr unsigned WARP = NS == 4 ? 0xffffffffu : 0xffffu;
    const float s2 = NS == 4 ? __shfl_sync(WARP, sum, COLS + cx) : 0.0f;
    if (c >= a.d) return;
    if (slot == 0) {
        const float g = weight(a.gate, c);
        if (a.dpost_w != nullptr) a.dpost_w[c] = g * sum;
        if (a.dpost_b != nullptr) a.dpost_b[c] = g * s2;
        if (a.dgate != nullptr) a.dgate[c] = a.post ? weight(a.post_w, c) * sum + offset(a.post_b, c) * s2 : sum;
    } else if (slot == NS / 2) {
        if (a.dw != nullptr) a.dw[c] = sum;
    } else if (slot == NS - 1) {
        if (a.db != nullptr) a.db[c] = sum;
    }
}

}  // namespace

cudaError_t launch_block_norm_params(const BlockNormArgs& a, int n, const float* part, cudaStream_t s) {
    const dim3 grid((a.d + COLS - 1) / COLS), block(COLS * SLOTS);
    return a.layer ? launch_pdl(block_norm_params_kernel<4>, grid, block, 0, s, a, n, part)
                   : launch_pdl(block_norm_params_kernel<2>, grid, block, 0, s, a, n, part);
}

size_t block_norm_bwd_floats(int R, int d, bool layer) {
    // whichever the operands' alignment lets it take
    return static_cast<size_t>(std::max({bwd_parts(R, d, BWD_SINGLE), bwd_parts(R, d, BWD_8), bwd_parts(R, d, BWD_16)})) * (layer ? 4 : 2) * d + (d > BWD_MAX_D ? 2 * static_cast<size_t>(R) : 0);
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
