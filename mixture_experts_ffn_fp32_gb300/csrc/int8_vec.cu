// 8-bit expert products on the integer dot-product instruction, for few rows
// per expert:
//   y[i, n] = sa[row] sb[e, n] sum_k a[row, k] b[e, n, k]     (sum exact, int32)
//   SwiGLU: h[i, n] = SiLU(y[i, n]) y[i, F + n], n < F = N / 2
//
// A warp takes four output channels (SwiGLU: two and their partners) and up to
// eight rows of one expert and walks the whole reduction, 512 values a step:
// the weights, which bound the product, are read once per eight rows, straight
// into registers, and each 16 bytes of them feed 4 dot products per row. The
// grid covers as many experts as can have rows; where that leaves SMs idle CTAs
// have fewer warps, and an expert's rows beyond eight go to further CTAs.
// Measured: one row, 4096 x 2048, 5.5 us (1.5 TB/s of weights: one round of loads
// and its latency); 64 rows of 256 experts, 4096 x 4096, 150 us (6.3 TB/s); from 32
// rows of one expert on the dot products bind (40 T operations/s).
#include <math_constants.h>

#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int WARPS = 8;
constexpr int NC = 4;  // weight rows per warp

struct VecParams {
    int M, Ma, K, N, E, slots;  // slots: experts that can have rows
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
    float sb[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        int n = SWIGLU ? n0 + (j >> 1) + (j & 1) * F : n0 + j;
        n = min(n, p.N - 1);  // channels past the end are read from the last and not stored
        const long long at = static_cast<long long>(e) * p.N + n;
        wr[j] = p.b + at * p.K;
        sb[j] = p.sb[at];
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
    // Bytes in flight for one row or two; for more, registers that leave room for a second
    // CTA (all four forms unrolled: 207 registers; 32 rows of 256 experts 111 -> 90 us,
    // 128 of 64, 65 -> 49, one row as before; 8 rows, 4096 x 4096, 12 -> 16).
#pragma unroll (RB == 1 ? 4 : RB == 2 ? 2 : 1)
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
                v = g * sigmoid_to<O>(g) * u;
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
    const int n0 = static_cast<int>(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * NO;
    pdl_wait();
    pdl_trigger();
    if (n0 >= F) return;
    if (static_cast<int>(blockIdx.y) == p.slots) {  // rows that no expert covers
        const int lo = min(max(p.offsets[p.E], 0), p.M);
        for (int i = lo + blockIdx.z; i < p.M; i += gridDim.z)
            if (lane < NO && n0 + lane < F)
                static_cast<O*>(p.out)[static_cast<long long>(i) * F + n0 + lane] = from_f32<O>(0.0f);
        return;
    }
    int e = 0, lo = 0, hi = p.M;
    if (p.offsets != nullptr) {
        // the blockIdx.y-th expert that has rows
        int before = 0;
        e = -1;
        for (int e0 = 0; e0 < p.E && e < 0; e0 += 32) {
            int a = 0, b = 0;
            if (e0 + lane < p.E) {
                a = min(max(p.offsets[e0 + lane], 0), p.M);
                b = min(max(p.offsets[e0 + lane + 1], a), p.M);
            }
            const unsigned some = __ballot_sync(0xffffffffu, b > a);
            const int want = static_cast<int>(blockIdx.y) - before;
            if (want < __popc(some)) {
                const bool mine = b > a && __popc(some & ((1u << lane) - 1)) == want;
                const int at = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
                e = e0 + at;
                lo = __shfl_sync(0xffffffffu, a, at);
                hi = __shfl_sync(0xffffffffu, b, at);
            }
            before += __popc(some);
        }
        if (e < 0) return;
    }
    for (int i = lo + 8 * blockIdx.z; i < hi; i += 8 * gridDim.z) {
        const int n = min(8, hi - i);
        if (n == 1) block<1, SWIGLU, O>(p, e, n0, i, n, lane);
        else if (n == 2) block<2, SWIGLU, O>(p, e, n0, i, n, lane);
        else if (n <= 4) block<4, SWIGLU, O>(p, e, n0, i, n, lane);
        else block<8, SWIGLU, O>(p, e, n0, i, n, lane);
    }
}

template <bool SWIGLU, typename O>
cudaError_t launch_t(const Int8Args& a, cudaStream_t s) {
    const int F = SWIGLU ? a.N / 2 : a.N, slots = a.E < a.M ? a.E : a.M;
    auto channel_ctas = [&](int w) { return (F + w * (SWIGLU ? NC / 2 : NC) - 1) / (w * (SWIGLU ? NC / 2 : NC)); };
    int warps = WARPS;
    while (warps > 2 && static_cast<long long>(channel_ctas(warps)) * slots < num_sms()) warps /= 2;
    const int gx = channel_ctas(warps);
    VecParams p{a.M, a.Ma, a.K, a.N, a.E, slots, a.lda, a.a, a.sa, a.b, a.sb, a.offsets, a.rows, a.out, a.err};
    // An expert's rows go over several CTAs, eight at a time, as far as that fills the SMs.
    const long long ctas = static_cast<long long>(gx) * slots;
    const int most = (a.M + 7) / 8, want = static_cast<int>((4LL * num_sms() + ctas - 1) / ctas);
    const int z = want < 1 ? 1 : want < most ? want : most;
    return launch_pdl(int8_vec_kernel<SWIGLU, O>, dim3(gx, slots + (a.offsets != nullptr ? 1 : 0), z), dim3(32 * warps),
                      0, s, p);
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
