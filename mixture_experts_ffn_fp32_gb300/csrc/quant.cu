// Rows to 8-bit integers with one scale each:
//   scale = max |x| / 127,  q = x / scale rounded to the nearest integer, ties
//   to even (the quotient exact, not its FP32 rounding)
// A row of zeros has scale 0; a row with an infinity or a NaN has q = 0 and
// scale NaN, which every product of the row then shows.
//
// Memory bound: x is read once into registers, by a warp for short rows and by
// a CTA else, while the CTA's next rows travel into shared memory, and q is
// written once. Measured, among other calls: 16384 x 2048 BF16 21 us (4.7 TB/s of
// 6.8; 24 alone with cold caches), FP32 32 us (5.3 TB/s); BF16 is held back by the
// instructions of exact rounding, 1100 a row, which keep 74 % of the issue slots busy
// (33 us when a branch sorted out what lies next to half steps: BF16 rows are full of
// it). Rows past 16384 are read twice, element by element: 4096 x 20480 BF16 124 us.
#include <math_constants.h>

#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int REG_MAX_K = 16384;  // 1024 threads x 16 elements
constexpr int DEPTH = 2;          // rows that travel ahead

template <int TPR>
MOE_DEV unsigned row_umax(unsigned v, unsigned* scratch, int& turn) {
    if constexpr (TPR < 32) {
#pragma unroll
        for (int o = TPR / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
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

// Largest |x| so far with a vector's: 16-bit types as pairs of integers, FP32 as
// an integer (an infinity's or a NaN's bits are the largest). row_bits turns it
// into FP32 bits.
template <typename T, int VEC>
MOE_DEV unsigned vec_umax(unsigned m, const Raw<T, VEC>& r) {
    if constexpr (VEC == 8) {
        constexpr unsigned M = 0x7fff7fffu;
        return __vimax3_u16x2(__vimax3_u16x2(m, r.v.x & M, r.v.y & M), r.v.z & M, r.v.w & M);
    } else {
        float f[VEC];
        r.get(f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) m = max(m, abs_bits(f[j]));
        return m;
    }
}
template <typename T, int VEC>
MOE_DEV unsigned row_bits(unsigned m) {
    if constexpr (VEC == 8) {
        const unsigned short h = static_cast<unsigned short>(max(m & 0xffffu, m >> 16));
        return abs_bits(to_f32(*reinterpret_cast<const T*>(&h)));
    }
    return m;
}

// What a row's largest |x| (as bits) makes of its elements.
struct RowScale {
    float scale, inv;
    int mode;  // 0: all zero, 1: FP32 arithmetic, 2: FP64 quotients
    MOE_DEV explicit RowScale(unsigned bits) {
        if (bits >= 0x7f800000u) {
            scale = CUDART_NAN_F;
            inv = 0.0f;
            mode = 0;
            return;
        }
        scale = __uint_as_float(bits) / 127.0f;
        // below this the reciprocal or a remainder could leave FP32's normal range
        mode = scale == 0.0f ? 0 : scale < 1e-30f ? 2 : 1;
        inv = mode == 1 ? 1.0f / scale : 0.0f;
    }
};

// A quotient of modes 0 and 2, out of line.
__device__ __noinline__ int quantize_rare(float x, float scale, int mode) {
    if (mode == 0) return 0;
    const double q = rint(static_cast<double>(x) / static_cast<double>(scale));
    return static_cast<int>(fmin(fmax(q, -127.0), 127.0));
}

// VEC quotients as bytes, rounded as the exact quotient rounds. BF16 rows are
// full of quotients next to half steps (the maximum over 127 is itself
// rounded), so no branch sorts them out:
//   t = x inv, t += (x - t scale) inv   the quotient rounded correctly: an exact half
//                                       step is met exactly and goes to the even side
//   y = t + 1.5 2^23                    the rounded integer q in y's low bits
//   e = x - q scale                     exact; |e| > scale / 2: t had rounded onto a
//                                       half step, and q is on the wrong side of it
template <int VEC>
MOE_DEV void quantize_vec(const RowScale& rs, const float (&v)[VEC], uint32_t (&b)[VEC]) {
    constexpr float MAGIC = 12582912.0f;
    const float half = 0.5f * rs.scale;
    auto settle = [&](float y, float e) {
        return __float_as_uint(fabsf(e) > half ? __fadd_rn(y, copysignf(1.0f, e)) : y);
    };
    if (rs.mode != 1) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) b[j] = static_cast<uint32_t>(quantize_rare(v[j], rs.scale, rs.mode));
    } else if constexpr (VEC > 1) {
        const F2 inv = f2(rs.inv, rs.inv), ns = f2(-rs.scale, -rs.scale), up = f2(MAGIC, MAGIC), dn = f2(-MAGIC, -MAGIC);
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
            const F2 x = f2(v[j], v[j + 1]);
            F2 t = mul2(x, inv);
            t = fma2(fma2(t, ns, x), inv, t);
            const F2 y = add2(t, up), e = fma2(add2(y, dn), ns, x);
            float ya, yb, ea, eb;
            unpack(y, ya, yb);
            unpack(e, ea, eb);
            b[j] = settle(ya, ea);
            b[j + 1] = settle(yb, eb);
        }
    } else {
        float t = v[0] * rs.inv;
        t = fmaf(fmaf(-t, rs.scale, v[0]), rs.inv, t);
        const float y = __fadd_rn(t, MAGIC);
        b[0] = settle(y, fmaf(-__fadd_rn(y, -MAGIC), rs.scale, v[0]));
    }
}
MOE_DEV uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

template <typename T, int VEC, int NV, int TPR>
struct Quant {
    static constexpr int THREADS = RowThreads<TPR>::THREADS;
    static constexpr int PER_SM = TPR == 1024 ? 1 : (VEC == 1 || NV * VEC > 16 ? 768 : 1024) / THREADS;
    using Fetch = RowFetch<T, VEC, NV, TPR, THREADS, DEPTH>;
};

template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(Quant<T, VEC, NV, TPR>::THREADS, Quant<T, VEC, NV, TPR>::PER_SM)
quantize_rows_kernel(int R, int K, const T* __restrict__ x, long long xs, int8_t* __restrict__ q,
                     float* __restrict__ scale) {
    using L = RowThreads<TPR>;
    __shared__ unsigned scratch[TPR > 32 ? 2 * (TPR / 32) : 1];
    const int t = L::col();
    const long long step = static_cast<long long>(gridDim.x) * L::ROWS;
    long long row = static_cast<long long>(blockIdx.x) * L::ROWS + L::row();
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
    for (; L::first(row) < R; row += step) {
        Raw<T, VEC> v[NV];
        unsigned m = 0;
        if constexpr (F::ASYNC) cp_async_wait<D - 1>();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = in.raw(slot, i);
            m = vec_umax(m, v[i]);
        }
        in.issue(slot, row + D * step, row + D * step < R);
        if constexpr (F::ASYNC) cp_async_commit();
        if (++slot == D) slot = 0;
        const RowScale rs(row_umax<TPR>(row_bits<T, VEC>(m), scratch, turn));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < K && row < R) {
                uint32_t b[VEC];
                float f[VEC];
                v[i].get(f);
                quantize_vec<VEC>(rs, f, b);
                int8_t* at = q + row * K + c;
                if constexpr (VEC == 8)
                    *reinterpret_cast<uint2*>(at) = make_uint2(pack4(b[0], b[1], b[2], b[3]), pack4(b[4], b[5], b[6], b[7]));
                else if constexpr (VEC == 4)
                    *reinterpret_cast<uint32_t*>(at) = pack4(b[0], b[1], b[2], b[3]);
                else
                    at[0] = static_cast<int8_t>(b[0]);
            }
        }
        if (t == 0 && row < R) scale[row] = rs.scale;
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
        for (int c = threadIdx.x; c < K; c += 1024) {
            const float v[1] = {to_f32(x[row * xs + c])};
            uint32_t b[1];
            quantize_vec<1>(rs, v, b);
            q[row * K + c] = static_cast<int8_t>(b[0]);
        }
        if (threadIdx.x == 0) scale[row] = rs.scale;
    }
}

template <typename T, int VEC, int NV, int TPR>
cudaError_t quant_t(const QuantArgs& a, cudaStream_t s) {
    using C = Quant<T, VEC, NV, TPR>;
    static bool done[64] = {};
    if (!allow_smem(quantize_rows_kernel<T, VEC, NV, TPR>, C::Fetch::SMEM, done)) return cudaErrorInvalidValue;
    return launch_pdl(quantize_rows_kernel<T, VEC, NV, TPR>, dim3(grid_rows(a.R, RowThreads<TPR>::ROWS, C::PER_SM)),
                      dim3(C::THREADS), C::Fetch::SMEM, s, a.R, a.K, static_cast<const T*>(a.x), a.x_stride, a.q, a.scale);
}

template <typename T, int VEC>
cudaError_t quant_v(const QuantArgs& a, cudaStream_t s) {
    constexpr bool SHORT = sizeof(T) == 2;
    if (a.K <= 8 * 16) return quant_t<T, VEC, 16 / VEC, 8>(a, s);
    if (a.K <= 32 * 16) return quant_t<T, VEC, 16 / VEC, 32>(a, s);
    // a warp without a sync beats a CTA of four (32768 rows of 1024, BF16: 19 against 26 us);
    // with 64 elements a lane it no longer does (16384 of 2048: 23 against 21 us)
    if constexpr (VEC > 1) {
        if (a.K <= 32 * 32) return quant_t<T, VEC, 32 / VEC, 32>(a, s);
    } else {
        if (a.K <= 128 * 8) return quant_t<T, 1, 8, 128>(a, s);
    }
    // three quarters of those of powers of two for 16-bit rows (BF16 of 2560, 100 MB: 43 -> 39
    // us; FP32 of 2880: 29 -> 37)
    if constexpr (SHORT)
        if (a.K <= 96 * 16) return quant_t<T, VEC, 16 / VEC, 96>(a, s);
    if (a.K <= 128 * 16) return quant_t<T, VEC, 16 / VEC, 128>(a, s);
    if constexpr (SHORT)
        if (a.K <= 192 * 16) return quant_t<T, VEC, 16 / VEC, 192>(a, s);
    if (a.K <= 256 * 16) return quant_t<T, VEC, 16 / VEC, 256>(a, s);
    if constexpr (SHORT)
        if (a.K <= 384 * 16) return quant_t<T, VEC, 16 / VEC, 384>(a, s);
    if (a.K <= 512 * 16) return quant_t<T, VEC, 16 / VEC, 512>(a, s);
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
