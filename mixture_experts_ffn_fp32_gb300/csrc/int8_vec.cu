// 8-bit expert products on the integer dot-product instruction, for few rows
// per expert:
//   y[i, n] = sa[row] sb[e, n] sum_k a[row, k] b[e, n, k]     (sum exact, int32)
//   SwiGLU: h[i, n] = SiLU(y[i, n]) y[i, F + n], n < F = N / 2
//
// A warp takes four output channels (SwiGLU: two and their partners) and up to
// eight rows of one expert and walks the whole reduction, 512 values a step:
// the weights, which bound the product, are read once per eight rows, straight
// into registers, and each 16 bytes of them feed 4 dot products per row.
#include <math_constants.h>

#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int WARPS = 8;
constexpr int NC = 4;  // weight rows per warp

struct VecParams {
    int M, Ma, K, N, E;
    long long lda;
    const int8_t* a;
    const float* sa;
    const int8_t* b;
    const float* sb;
    const int32_t* offsets;
    const int32_t* rows;
    void* out;
    int* err;
};

template <int RB, bool SWIGLU, typename O>
MOE_DEV void block(const VecParams& p, int e, int n0, int i0, int nrows, int lane) {
    const int F = SWIGLU ? p.N / 2 : p.N;
    constexpr int NO = SWIGLU ? NC / 2 : NC;  // outputs per row
    const int8_t* wr[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        int n = SWIGLU ? n0 + (j >> 1) + (j & 1) * F : n0 + j;
        n = min(n, p.N - 1);  // channels past the end are read from the last and not stored
        wr[j] = p.b + (static_cast<long long>(e) * p.N + n) * p.K;
    }
    const int8_t* ar[RB];
    float sa[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        int src = i0 + min(r, nrows - 1);
        bool ok = true;
        if (p.rows != nullptr) {
            src = p.rows[src];
            ok = src >= 0 && src < p.Ma;
            if (!ok) {
                if (lane == 0) atomicOr(p.err, ERRBIT_INDEX);
                src = 0;
            }
        }
        ar[r] = p.a + src * p.lda;
        sa[r] = ok ? p.sa[src] : CUDART_NAN_F;
    }
    int acc[RB][NC] = {};
    for (int k = lane * 16; k < p.K; k += 512) {
        int4 w[NC], x[RB];
#pragma unroll
        for (int j = 0; j < NC; ++j) w[j] = __ldg(reinterpret_cast<const int4*>(wr[j] + k));
#pragma unroll
        for (int r = 0; r < RB; ++r) x[r] = __ldg(reinterpret_cast<const int4*>(ar[r] + k));
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                acc[r][j] = __dp4a(x[r].x, w[j].x, acc[r][j]);
                acc[r][j] = __dp4a(x[r].y, w[j].y, acc[r][j]);
                acc[r][j] = __dp4a(x[r].z, w[j].z, acc[r][j]);
                acc[r][j] = __dp4a(x[r].w, w[j].w, acc[r][j]);
            }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int j = 0; j < NC; ++j) acc[r][j] = __reduce_add_sync(0xffffffffu, acc[r][j]);
    float sb[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        int n = SWIGLU ? n0 + (j >> 1) + (j & 1) * F : n0 + j;
        sb[j] = p.sb[static_cast<long long>(e) * p.N + min(n, p.N - 1)];
    }
    // lane r * NO + j stores output j of row r
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            if (lane != (r * NO + j) || r >= nrows || n0 + j >= F) continue;
            float v;
            if (SWIGLU) {
                const float g = static_cast<float>(acc[r][2 * j]) * sa[r] * sb[2 * j];
                const float u = static_cast<float>(acc[r][2 * j + 1]) * sa[r] * sb[2 * j + 1];
                v = g * sigmoid_f(g) * u;
            } else {
                v = static_cast<float>(acc[r][j]) * sa[r] * sb[j];
            }
            static_cast<O*>(p.out)[static_cast<long long>(i0 + r) * F + n0 + j] = from_f32<O>(v);
        }
}

template <bool SWIGLU, typename O>
__global__ void __launch_bounds__(32 * WARPS)
int8_vec_kernel(const VecParams p) {
    const int lane = static_cast<int>(lane_id());
    const int F = SWIGLU ? p.N / 2 : p.N;
    constexpr int NO = SWIGLU ? NC / 2 : NC;
    const int n0 = (blockIdx.x * WARPS + (threadIdx.x >> 5)) * NO;
    pdl_wait();
    pdl_trigger();
    if (n0 >= F) return;
    const int e = static_cast<int>(blockIdx.y);
    if (e == p.E) {  // rows that no expert covers
        const int lo = min(max(p.offsets[p.E], 0), p.M);
        for (int i = lo; i < p.M; ++i)
            if (lane < NO && n0 + lane < F)
                static_cast<O*>(p.out)[static_cast<long long>(i) * F + n0 + lane] = from_f32<O>(0.0f);
        return;
    }
    int lo = 0, hi = p.M;
    if (p.offsets != nullptr) {
        lo = min(max(p.offsets[e], 0), p.M);
        hi = min(max(p.offsets[e + 1], lo), p.M);
    }
    for (int i = lo; i < hi; i += 8) {
        const int n = min(8, hi - i);
        if (n == 1) block<1, SWIGLU, O>(p, e, n0, i, n, lane);
        else if (n == 2) block<2, SWIGLU, O>(p, e, n0, i, n, lane);
        else if (n <= 4) block<4, SWIGLU, O>(p, e, n0, i, n, lane);
        else block<8, SWIGLU, O>(p, e, n0, i, n, lane);
    }
}

template <bool SWIGLU, typename O>
cudaError_t launch_t(const Int8Args& a, cudaStream_t s) {
    const int F = SWIGLU ? a.N / 2 : a.N, per = WARPS * (SWIGLU ? NC / 2 : NC);
    VecParams p{a.M, a.Ma, a.K, a.N, a.E, a.lda, a.a, a.sa, a.b, a.sb, a.offsets, a.rows, a.out, a.err};
    return launch_pdl(int8_vec_kernel<SWIGLU, O>, dim3((F + per - 1) / per, a.E + (a.offsets != nullptr ? 1 : 0)),
                      dim3(32 * WARPS), 0, s, p);
}

}  // namespace

cudaError_t launch_int8_vec(const Int8Args& a, cudaStream_t s) {
    switch (a.out_dtype) {
        case MOE_BF16: return a.swiglu ? launch_t<true, __nv_bfloat16>(a, s) : launch_t<false, __nv_bfloat16>(a, s);
        case MOE_F16: return a.swiglu ? launch_t<true, __half>(a, s) : launch_t<false, __half>(a, s);
        default: return a.swiglu ? launch_t<true, float>(a, s) : launch_t<false, float>(a, s);
    }
}

}  // namespace moe
