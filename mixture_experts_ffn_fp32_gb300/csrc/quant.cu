// Rows to 8-bit integers with one scale each:
//   scale = max |x| / 127,  q = x / scale rounded to the nearest integer, ties
//   to even (the quotient exact, not its FP32 rounding)
// A row of zeros has scale 0; a row with an infinity or a NaN has q = 0 and
// scale NaN, which every product of the row then shows.
//
// Memory bound: x is read once into registers, by a warp for short rows and by
// a CTA else, while the CTA's next rows travel into shared memory, and q is
// written once.
#include <math_constants.h>

#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int REG_MAX_K = 16384;  // 1024 threads x 16 elements
constexpr int DEPTH = 2;          // rows that travel ahead

template <int TPR>
MOE_DEV unsigned row_umax(unsigned v, unsigned* scratch, int& turn) {
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        unsigned* s = scratch + (turn & 1) * W;
        ++turn;
        if (lane_id() == 0) s[threadIdx.x >> 5] = v;
        __syncthreads();
        v = __reduce_max_sync(0xffffffffu, lane_id() < W ? s[lane_id()] : 0u);
    }
    return v;
}

MOE_DEV unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// What a row's largest |x| (as bits) makes of its elements.
struct RowScale {
    float scale, inv;
    int mode;  // 0: all zero, 1: FP32 quotient with an exact remainder, 2: FP64 quotient
    MOE_DEV explicit RowScale(unsigned bits) {
        if (bits >= 0x7f800000u) {
            scale = CUDART_NAN_F;
            inv = 0.0f;
            mode = 0;
            return;
        }
        scale = __uint_as_float(bits) / 127.0f;
        // below this the reciprocal or the remainder could leave FP32's normal range
        mode = scale == 0.0f ? 0 : scale < 1e-30f ? 2 : 1;
        inv = mode == 1 ? 1.0f / scale : 0.0f;
    }
    MOE_DEV int quantize(float x) const {
        if (mode == 1) {
            const float t = x * inv;  // off by at most 2^-23 of itself: 2e-5 at 127
            float q = rintf(t);
            if (fabsf(t - q) > 0.4999f) {
                // x - q scale is exact in FP32 (q has 7 bits and the difference is at
                // most a little over half a step); it says on which side x lies
                const float rem = fmaf(-q, scale, x), half = 0.5f * scale;
                const bool odd = (static_cast<int>(q) & 1) != 0;
                if (rem > half || (rem == half && odd)) q += 1.0f;
                else if (rem < -half || (rem == -half && odd)) q -= 1.0f;
            }
            return static_cast<int>(q);
        }
        if (mode == 0) return 0;
        const double q = rint(static_cast<double>(x) / static_cast<double>(scale));
        return static_cast<int>(fmin(fmax(q, -127.0), 127.0));
    }
};

// VEC quotients as bytes. Adding 1.5 2^23 leaves the rounded integer in a
// float's low bits; what lies within 1e-4 of a half step, or has no FP32
// quotient, is decided one by one.
template <int VEC>
MOE_DEV void quantize_vec(const RowScale& rs, const float (&v)[VEC], uint32_t (&b)[VEC]) {
    constexpr float MAGIC = 12582912.0f;
    bool edge = rs.mode != 1;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const float t = v[j] * rs.inv, y = __fadd_rn(t, MAGIC), q = __fadd_rn(y, -MAGIC);
        edge = edge || fabsf(t - q) > 0.4999f;
        b[j] = __float_as_uint(y);
    }
    if (edge) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) b[j] = static_cast<uint32_t>(rs.quantize(v[j]));
    }
}
MOE_DEV uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

template <typename T, int VEC, int NV, int TPR>
struct Quant {
    static constexpr int THREADS = TPR == 32 ? 128 : TPR;
    static constexpr int PER_SM = TPR == 1024 ? 1 : (VEC == 1 || NV * VEC > 16 ? 768 : 1024) / THREADS;
    using Fetch = RowFetch<T, VEC, NV, TPR, THREADS, DEPTH>;
};

template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(Quant<T, VEC, NV, TPR>::THREADS, Quant<T, VEC, NV, TPR>::PER_SM)
quantize_rows_kernel(int R, int K, const T* __restrict__ x, long long xs, int8_t* __restrict__ q,
                     float* __restrict__ scale) {
    constexpr int RPC = TPR == 32 ? 4 : 1;
    __shared__ unsigned scratch[TPR > 32 ? 2 * (TPR / 32) : 1];
    const int t = TPR == 32 ? static_cast<int>(lane_id()) : static_cast<int>(threadIdx.x);
    const long long step = static_cast<long long>(gridDim.x) * RPC;
    long long row = static_cast<long long>(blockIdx.x) * RPC + (TPR == 32 ? threadIdx.x >> 5 : 0);
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    using F = typename Quant<T, VEC, NV, TPR>::Fetch;
    constexpr int D = F::D;
    extern __shared__ __align__(16) uint8_t smem[];
    F in;
    in.init(smem, x, xs, K, t);
#pragma unroll
    for (int s = 0; s < D; ++s) {
        in.issue(s, row + s * step, row + s * step < R);
        if constexpr (F::ASYNC) cp_async_commit();
    }
    int slot = 0;
    for (; row < R; row += step) {
        float v[NV][VEC];
        unsigned m = 0;
        if constexpr (F::ASYNC) cp_async_wait<D - 1>();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            in.get(slot, i, v[i]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) m = max(m, abs_bits(v[i][j]));
        }
        in.issue(slot, row + D * step, row + D * step < R);
        if constexpr (F::ASYNC) cp_async_commit();
        if (++slot == D) slot = 0;
        const RowScale rs(row_umax<TPR>(m, scratch, turn));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < K) {
                uint32_t b[VEC];
                quantize_vec<VEC>(rs, v[i], b);
                int8_t* at = q + row * K + c;
                if constexpr (VEC == 8)
                    *reinterpret_cast<uint2*>(at) = make_uint2(pack4(b[0], b[1], b[2], b[3]), pack4(b[4], b[5], b[6], b[7]));
                else if constexpr (VEC == 4)
                    *reinterpret_cast<uint32_t*>(at) = pack4(b[0], b[1], b[2], b[3]);
                else
                    at[0] = static_cast<int8_t>(b[0]);
            }
        }
        if (t == 0) scale[row] = rs.scale;
    }
}

// Rows longer than the registers hold: two passes, the second from L2.
template <typename T>
__global__ void __launch_bounds__(1024)
quantize_rows_long_kernel(int R, int K, const T* __restrict__ x, long long xs, int8_t* __restrict__ q,
                          float* __restrict__ scale) {
    __shared__ unsigned scratch[2 * 32];
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    for (long long row = blockIdx.x; row < R; row += gridDim.x) {
        unsigned m = 0;
        for (int c = threadIdx.x; c < K; c += 1024) m = max(m, abs_bits(to_f32(x[row * xs + c])));
        const RowScale rs(row_umax<1024>(m, scratch, turn));
        for (int c = threadIdx.x; c < K; c += 1024)
            q[row * K + c] = static_cast<int8_t>(rs.quantize(to_f32(x[row * xs + c])));
        if (threadIdx.x == 0) scale[row] = rs.scale;
    }
}

template <typename T, int VEC, int NV, int TPR>
cudaError_t quant_t(const QuantArgs& a, cudaStream_t s) {
    using C = Quant<T, VEC, NV, TPR>;
    static bool done[64] = {};
    if (!allow_smem(quantize_rows_kernel<T, VEC, NV, TPR>, C::Fetch::SMEM, done)) return cudaErrorInvalidValue;
    return launch_pdl(quantize_rows_kernel<T, VEC, NV, TPR>, dim3(grid_rows(a.R, TPR == 32 ? 4 : 1, C::PER_SM)),
                      dim3(C::THREADS), C::Fetch::SMEM, s, a.R, a.K, static_cast<const T*>(a.x), a.x_stride, a.q, a.scale);
}

template <typename T, int VEC>
cudaError_t quant_v(const QuantArgs& a, cudaStream_t s) {
    if (a.K <= 32 * 8) return quant_t<T, VEC, 8 / VEC, 32>(a, s);
    if (a.K <= 32 * 32) return quant_t<T, VEC, 32 / VEC, 32>(a, s);
    if (a.K <= 128 * 16) return quant_t<T, VEC, 16 / VEC, 128>(a, s);
    if (a.K <= 256 * 16) return quant_t<T, VEC, 16 / VEC, 256>(a, s);
    return quant_t<T, VEC, 16 / VEC, 1024>(a, s);
}

template <typename T>
cudaError_t quant_d(const QuantArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (a.K > REG_MAX_K)
        return launch_pdl(quantize_rows_long_kernel<T>, dim3(grid_rows(a.R, 1, 2)), dim3(1024), 0, s, a.R, a.K,
                          static_cast<const T*>(a.x), a.x_stride, a.q, a.scale);
    const bool vec = a.K % V == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 &&
                     (a.x_stride * static_cast<long long>(sizeof(T))) % 16 == 0 &&
                     (reinterpret_cast<uintptr_t>(a.q) & 7u) == 0;
    return vec ? quant_v<T, V>(a, s) : quant_v<T, 1>(a, s);
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantArgs& a, cudaStream_t s) {
    switch (a.dtype) {
        case MOE_BF16: return quant_d<__nv_bfloat16>(a, s);
        case MOE_F16: return quant_d<__half>(a, s);
        default: return quant_d<float>(a, s);
    }
}

}  // namespace moe
