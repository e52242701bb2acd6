// The norms on both sides of a block, fused with its gate and the residual:
//
//   z  = Norm(y; wp, bp) or y          y: the block's output
//   x' = alpha x + g z                 g: 1, a vector [d], or a value per element
//   n  = Norm(x'; w, b)                the next block's input
//   Norm(v; w, b) = (v - mu) r w + b,  r = 1 / sqrt(mean((v - mu)^2) + eps), mu = mean(v) (RMS: 0)
//
// Backward, from dn, dx' and the forward's x', y and statistics:
//   h = dn w,  xh = (x' - mu) r,       t = dx' + r (h - [mean(h)] - xh mean(h xh))
//   dx = alpha t,  dg = t z (summed over the rows of a vector)
//   k = t g wp,  yh = (y - muy) ry,    dy = ry (k - [mean(k)] - yh mean(k yh))   (without a norm: t g)
//   dwp = sum t g yh,  dbp = sum t g,  dw = sum dn xh,  db = sum dn       ([.]: layer norm alone)
// The parameters' gradients come from four column sums: S1 = sum t yh, S2 = sum t (with a
// gate per element: of t g), S3 = sum dn xh, S4 = sum dn.
//
// Statistics and sums are FP32; n is taken of x' before its rounding.
//
// Both directions are bound by memory: the forward reads x, y (and a gate per element) and writes x'
// and n, the backward reads dn, dx', x', y and writes dx and dy, each element once. A row is in the
// registers of part of a warp (short rows) or of a CTA from its loads to its outputs, the next row
// under way; a CTA meets once for each sum over the row (y's and x''s statistics; backward h xh, k yh),
// so several share an SM. The columns' sums stay in registers until a CTA's rows are done, then one
// partial row a CTA goes through memory (no atomics: bit-reproducible).
//
// Measured (one GB300, 6.8 TB/s copy rate; a plain copy of as many bytes takes a tenth more than that
// at these sizes): forward, 16384 x 2048 BF16, RMS, 45 us (6.0 TB/s), layer norm 56; 8192 x 4096 FP32
// layer norm 83 (6.5 TB/s). Backward with its column sums, 8192 x 4096 BF16 RMS 68 us (5.9 TB/s), layer
// norm 99 (four column sums fill the registers, 8 columns a thread); 8192 x 2048 FP32 65 (6.2 TB/s).
// Rows on no 16 bytes, element by element: 20000 x 1411 BF16 69 us (3.3 TB/s), backward of 10000 71.
// Few rows are latency: 128 x 4096 4 us. What counts most is L1: it holds what is neither in registers
// nor in shared memory (vectors, spilled sums), and more rows ahead take it away (see Ahead).
#pragma once

#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int LONG_THREADS = 1024;

template <typename T>
struct Io {
    const T *x, *y, *g, *dn, *dxo;  // g: a gate per element
    T *out, *n, *dy, *dgate;        // out: x' or dx
};
template <typename T>
Io<T> io_of(const BlockNormArgs& a) {
    return {static_cast<const T*>(a.x), static_cast<const T*>(a.y), static_cast<const T*>(a.gate_elem),
            static_cast<const T*>(a.dn), static_cast<const T*>(a.dxo), static_cast<T*>(a.out), static_cast<T*>(a.n),
            static_cast<T*>(a.dy), static_cast<T*>(a.dgate_elem)};
}

// Where the statistics of row r stand: RMS [2, R] (of y, of x'), layer [4, R] (mean and rstd of each).
MOE_DEV float* stat(const BlockNormArgs& a, int which, int r) {
    return a.stats + static_cast<long long>(a.layer ? which : which >> 1) * a.R + r;
}

MOE_DEV float weight(const float* w, int c) { return w != nullptr ? __ldg(w + c) : 1.0f; }
MOE_DEV float offset(const float* b, int c) { return b != nullptr ? __ldg(b + c) : 0.0f; }

// Mean (RMS: 0) and 1 / deviation of the row value(0 .. d - 1), by a CTA.
template <typename V>
MOE_DEV void long_stats(V value, int d, bool layer, float eps, float* scratch, int& turn, float& mean, float& rstd) {
    float m0 = 0.0f, unused = 0.0f;
    if (layer) {
        for (int c = threadIdx.x; c < d; c += LONG_THREADS) m0 += value(c);
        row_sum2<LONG_THREADS>(m0, unused, scratch, turn);
        m0 /= static_cast<float>(d);
    }
    float r1 = 0.0f, r2 = 0.0f;
    for (int c = threadIdx.x; c < d; c += LONG_THREADS) {
        const float v = value(c) - m0;
        r1 += v;
        r2 += v * v;
    }
    row_sum2<LONG_THREADS>(r1, r2, scratch, turn);
    const float rest = layer ? r1 / static_cast<float>(d) : 0.0f;  // what rounding left in m0
    rstd = rstd_of(r2 / static_cast<float>(d) - rest * rest, eps);
    mean = joined(m0, rest);
}

template <typename T>
__global__ void __launch_bounds__(LONG_THREADS) block_norm_long_kernel(const __grid_constant__ BlockNormArgs a, Io<T> p) {
    __shared__ float scratch[4 * 32];
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    for (int row = blockIdx.x; row < a.R; row += gridDim.x) {
        const T* x = p.x + row * a.x_stride;
        const T* y = p.y != nullptr ? p.y + row * a.y_stride : nullptr;
        const T* g = p.g != nullptr ? p.g + row * a.gate_stride : nullptr;
        float ym = 0.0f, yr = 1.0f, xm = 0.0f, xr = 1.0f;
        if (a.post)
            long_stats([&](int c) { return to_f32(y[c]); }, a.d, a.layer, a.eps, scratch, turn, ym, yr);
        auto stream = [&](int c) {
            if (y == nullptr) return to_f32(x[c]);
            float z = to_f32(y[c]);
            if (a.post) z = (z - ym) * yr * weight(a.post_w, c) + offset(a.post_b, c);
            const float gc = g != nullptr ? to_f32(g[c]) : weight(a.gate, c);
            return a.alpha * to_f32(x[c]) + gc * z;
        };
        if (p.n != nullptr) long_stats(stream, a.d, a.layer, a.eps, scratch, turn, xm, xr);
        for (int c = threadIdx.x; c < a.d; c += LONG_THREADS) {
            const float v = stream(c);
            if (p.out != nullptr) p.out[static_cast<long long>(row) * a.d + c] = from_f32<T>(v);
            if (p.n != nullptr)
                p.n[static_cast<long long>(row) * a.d + c] = from_f32<T>((v - xm) * xr * weight(a.w, c) + offset(a.b, c));
        }
        if (threadIdx.x == 0 && a.stats != nullptr) {
            if (a.layer) {
                *stat(a, 0, row) = ym;
                *stat(a, 2, row) = xm;
            }
            *stat(a, 1, row) = yr;
            *stat(a, 3, row) = xr;
        }
    }
}

// A row's t at column c from the row's sums of h and h xh over d.
template <typename T>
struct RowGrad {
    const T *x, *y, *g, *dn, *dxo;
    float ym, yr, xm, xr, m1, m2;
    MOE_DEV RowGrad(const BlockNormArgs& a, const Io<T>& p, int row) {
        x = p.x + row * a.x_stride;
        y = p.y != nullptr ? p.y + row * a.y_stride : nullptr;
        g = p.g != nullptr ? p.g + row * a.gate_stride : nullptr;
        dn = p.dn != nullptr ? p.dn + row * a.dn_stride : nullptr;
        dxo = p.dxo != nullptr ? p.dxo + row * a.dxo_stride : nullptr;
        ym = xm = m1 = m2 = 0.0f;
        yr = xr = 1.0f;
        if (a.post) {
            if (a.layer) ym = *stat(a, 0, row);
            yr = *stat(a, 1, row);
        }
        if (dn != nullptr) {
            if (a.layer) xm = *stat(a, 2, row);
            xr = *stat(a, 3, row);
        }
    }
    MOE_DEV float xh(int c) const { return (to_f32(x[c]) - xm) * xr; }
    MOE_DEV float h(const BlockNormArgs& a, int c) const { return to_f32(dn[c]) * weight(a.w, c); }
    MOE_DEV float t(const BlockNormArgs& a, int c) const {
        float v = dxo != nullptr ? to_f32(dxo[c]) : 0.0f;
        if (dn != nullptr) v += xr * (h(a, c) - m1 - xh(c) * m2);
        return v;
    }
    MOE_DEV float yh(int c) const { return (to_f32(y[c]) - ym) * yr; }
    MOE_DEV float gate(const BlockNormArgs& a, int c) const { return g != nullptr ? to_f32(g[c]) : weight(a.gate, c); }
};

// m12 [R, 2]: the rows' means of h and h xh, for the columns' pass.
template <typename T>
__global__ void __launch_bounds__(LONG_THREADS)
block_norm_bwd_long_kernel(const __grid_constant__ BlockNormArgs a, Io<T> p, float* m12) {
    __shared__ float scratch[4 * 32];
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    const float inv_d = 1.0f / static_cast<float>(a.d);
    for (int row = blockIdx.x; row < a.R; row += gridDim.x) {
        RowGrad<T> r(a, p, row);
        if (r.dn != nullptr) {
            float s1 = 0.0f, s2 = 0.0f;
            for (int c = threadIdx.x; c < a.d; c += LONG_THREADS) {
                const float h = r.h(a, c);
                s1 += h;
                s2 += h * r.xh(c);
            }
            row_sum2<LONG_THREADS>(s1, s2, scratch, turn);
            r.m1 = a.layer ? s1 * inv_d : 0.0f;
            r.m2 = s2 * inv_d;
        }
        if (threadIdx.x == 0 && m12 != nullptr) {
            m12[2 * row] = r.m1;
            m12[2 * row + 1] = r.m2;
        }
        float k1 = 0.0f, k2 = 0.0f;
        if (a.post) {
            for (int c = threadIdx.x; c < a.d; c += LONG_THREADS) {
                const float k = r.t(a, c) * r.gate(a, c) * weight(a.post_w, c);
                k1 += k;
                k2 += k * r.yh(c);
            }
            row_sum2<LONG_THREADS>(k1, k2, scratch, turn);
            k1 = a.layer ? k1 * inv_d : 0.0f;
            k2 *= inv_d;
        }
        const long long o = static_cast<long long>(row) * a.d;
        for (int c = threadIdx.x; c < a.d; c += LONG_THREADS) {
            const float t = r.t(a, c);
            p.out[o + c] = from_f32<T>(a.alpha * t);
            if (r.y == nullptr) continue;
            const float tg = t * r.gate(a, c);
            float dy = tg;
            if (a.post) dy = r.yr * (tg * weight(a.post_w, c) - k1 - r.yh(c) * k2);
            p.dy[o + c] = from_f32<T>(dy);
            if (p.dgate != nullptr) {
                float z = to_f32(r.y[c]);
                if (a.post) z = r.yh(c) * weight(a.post_w, c) + offset(a.post_b, c);
                p.dgate[o + c] = from_f32<T>(t * z);
            }
        }
    }
}

// part [gridDim.y][RMS: S1, S3; layer: S1 .. S4][d]
template <typename T>
__global__ void __launch_bounds__(256)
block_norm_bwd_cols_kernel(const __grid_constant__ BlockNormArgs a, Io<T> p, const float* __restrict__ m12, float* part) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (c >= a.d) return;
    float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f, s4 = 0.0f;
    for (int row = blockIdx.y; row < a.R; row += gridDim.y) {
        RowGrad<T> r(a, p, row);
        r.m1 = m12[2 * row];
        r.m2 = m12[2 * row + 1];
        if (r.dn != nullptr) {
            const float dn = to_f32(r.dn[c]);
            s3 += dn * r.xh(c);
            s4 += dn;
        }
        if (r.y != nullptr) {
            const float t = r.t(a, c) * (r.g != nullptr ? to_f32(r.g[c]) : 1.0f);
            s1 += t * r.yh(c);
            s2 += t;
        }
    }
    float* o = part + static_cast<long long>(blockIdx.y) * (a.layer ? 4 : 2) * a.d + c;
    o[0] = s1;
    if (a.layer) {
        o[a.d] = s2;
        o[2 * a.d] = s3;
        o[3 * a.d] = s4;
    } else {
        o[a.d] = s3;
    }
}

// ---------------------------------------------------------------------------
// rows held in registers
// ---------------------------------------------------------------------------
// Longest rows held in registers (backward: with their columns' sums).
constexpr int FWD_MAX_D = 16384;
constexpr int BWD_MAX_D = 8192;

// A thread's columns of a vector as pairs, `none` where there is no vector, zeros past the row's end.
template <int VEC, int NV, int TPR>
MOE_DEV void columns(const float* p, float none, int d, int t, F2 (&o)[NV * VEC / 2]) {
    float f[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[i][j] = c < d ? none : 0.0f;
        if (c < d && p != nullptr) load_f32<VEC>(p + c, f[i]);
    }
#pragma unroll
    for (int k = 0; k < NV * VEC / 2; ++k) o[k] = f2(f[2 * k / VEC][2 * k % VEC], f[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
}

// A thread's columns of a vector in its own part of shared memory, 4 at a time.
struct alignas(16) F4 {
    F2 a, b;
};
template <int N2, int THREADS>
MOE_DEV void keep(F4* slots, const F2 (&v)[N2]) {
#pragma unroll
    for (int k = 0; k < N2; k += 2) slots[k / 2 * THREADS + threadIdx.x] = F4{v[k], v[k + 1]};
}
template <int N2, int THREADS>
MOE_DEV void kept(const F4* slots, F2 (&v)[N2]) {
#pragma unroll
    for (int k = 0; k < N2; k += 2) {
        const F4 f = slots[k / 2 * THREADS + threadIdx.x];
        v[k] = f.a;
        v[k + 1] = f.b;
    }
}

template <int N2>
MOE_DEV void same(const F2 (&regs)[N2], F2 (&v)[N2]) {
#pragma unroll
    for (int k = 0; k < N2; ++k) v[k] = regs[k];
}

// A thread's columns of a row to memory, each rounded once.
template <typename T, int VEC, int NV, int TPR>
MOE_DEV void put(T* row, int d, int t, const F2 (&v)[NV * VEC / 2]) {
    float f[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV * VEC / 2; ++k) unpack(v[k], f[2 * k / VEC][2 * k % VEC], f[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * VEC;
        if (c < d) {
            Raw<T, VEC> out;
            out.set(f[i]);
            out.store(row + c);
        }
    }
}

// Statistics of a row held as pairs. Layer: leaves v - m and what is still to be added (shift).
template <int VEC, int NV, int TPR, bool LAYER>
MOE_DEV void row_stats(F2 (&v)[NV * VEC / 2], int d, int t, float inv_d, float eps, float4* scratch, int& turn, float& mean,
                       float& shift, float& rstd) {
    if constexpr (LAYER) {
        float var;
        row_moments<VEC, NV, TPR>(v, d, t, inv_d, scratch, turn, mean, shift, var);
        rstd = rstd_of(var, eps);
    } else {
        F2 q2 = mul2(v[0], v[0]);
#pragma unroll
        for (int k = 1; k < NV * VEC / 2; ++k) q2 = fma2(v[k], v[k], q2);
        float q = both(q2);
        row_sum<TPR>(q, reinterpret_cast<float*>(scratch), turn);
        rstd = rstd_of(q * inv_d, eps);
        mean = shift = 0.0f;
    }
}

// A thread's columns of one operand's next row, under way while it works on this one: in
// shared memory (RowFetch), or in registers where elements are too short for cp.async. One row
// ahead is enough, and what more shared memory would take from L1 is missed there by the
// vectors (backward of 16384 x 2048 BF16: 86 us one row ahead, 146 two; forward 43, 49).
template <typename T, int VEC, int NV, int TPR>
using Ahead = RowFetch<T, VEC, NV, TPR, RowThreads<TPR>::THREADS, 1>;

template <typename T, int VEC, int NV, int TPR, bool LAYER>
struct Forward {
    static constexpr int THREADS = RowThreads<TPR>::THREADS;
    static constexpr int COLS = NV * VEC;
    // CTAs of an SM: as many threads as the registers of a thread's columns leave
    static constexpr int PER_SM = (TPR == 1024 || COLS <= 8 ? 1024 : TPR == 512 || LAYER ? 512 : 768) / THREADS;
    using Fetch = Ahead<T, VEC, NV, TPR>;
    // Where a thread's columns of the vectors (the gate times wp and bp, w, b) are: in registers with
    // 16 columns and few or 16-bit operands, else in its own part of shared memory, or fetched for each
    // row where neither has room (us, registers : shared memory, 134 MB in and out: 16384 x 2048 BF16
    // 45 : 46, layer norm 56 : 60; 8192 x 4096 47 : 43, layer norm 59 : 64, FP32 91 : 83; 8 columns:
    // 20000 x 1411 BF16 85 : 69, 200000 x 128 60 : 56).
    static constexpr bool REGS = VEC > 1 && COLS == 16 && (LAYER ? sizeof(T) == 2 && TPR < 1024 : TPR <= 128);
    static constexpr bool KEPT = !REGS && COLS * THREADS <= 8192;
    static constexpr int VECTOR = COLS * 4 * THREADS, VECTORS = !KEPT ? 0 : LAYER ? 4 : 2;  // bytes of one
    static constexpr int smem(int operands) { return VECTORS * VECTOR + operands * Fetch::SMEM; }
};

template <typename T, int VEC, int NV, int TPR, bool LAYER>
__global__ void __launch_bounds__(Forward<T, VEC, NV, TPR, LAYER>::THREADS, Forward<T, VEC, NV, TPR, LAYER>::PER_SM)
block_norm_kernel(const __grid_constant__ BlockNormArgs a, const __grid_constant__ Io<T> p) {
    using F = typename Forward<T, VEC, NV, TPR, LAYER>::Fetch;
    using L = RowThreads<TPR>;
    constexpr int N2 = NV * VEC / 2;
    using C = Forward<T, VEC, NV, TPR, LAYER>;
    constexpr int THREADS = C::THREADS;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float4 scratch[TPR > 32 ? 2 * (TPR / 32) : 1];
    const int t = L::col(), d = a.d;
    const long long step = static_cast<long long>(gridDim.x) * L::ROWS;
    long long row = static_cast<long long>(blockIdx.x) * L::ROWS + L::row();
    const float inv_d = 1.0f / static_cast<float>(d);
    const bool block = p.y != nullptr, post = a.post != 0, norm = p.n != nullptr, elem = p.g != nullptr;
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    F fx, fy, fg;
    F4* const sgw = reinterpret_cast<F4*>(smem);  // then w, and of layer norms the two offsets
    F4* const sw = sgw + C::VECTOR / 16;
    F4* const sgb = sw + C::VECTOR / 16;
    F4* const sb = sgb + C::VECTOR / 16;
    uint8_t* const ahead = smem + C::VECTORS * C::VECTOR;
    fx.init(ahead, p.x, a.x_stride, d, t);
    fy.init(ahead + F::SMEM, p.y, a.y_stride, d, t);
    fg.init(ahead + 2 * F::SMEM, p.g, a.gate_stride, d, t);
    if (block) fy.issue(0, row, row < a.R);
    cp_async_commit();
    fx.issue(0, row, row < a.R);
    if (elem) fg.issue(0, row, row < a.R);
    cp_async_commit();
    // z = yh wp + bp; a gate per channel is taken into both
    auto post_vector = [&](const float* p, float none, F2 (&v)[N2]) {
        F2 g[N2];
        columns<VEC, NV, TPR>(a.gate, 1.0f, d, t, g);
        columns<VEC, NV, TPR>(p, none, d, t, v);
#pragma unroll
        for (int k = 0; k < N2; ++k) v[k] = mul2(v[k], g[k]);
    };
    F2 rgw[C::REGS ? N2 : 1], rw[C::REGS ? N2 : 1], rgb[C::REGS && LAYER ? N2 : 1], rb[C::REGS && LAYER ? N2 : 1];
    if constexpr (C::REGS) {
        post_vector(a.post_w, 1.0f, rgw);
        columns<VEC, NV, TPR>(a.w, 1.0f, d, t, rw);
        if constexpr (LAYER) {
            post_vector(a.post_b, 0.0f, rgb);
            columns<VEC, NV, TPR>(a.b, 0.0f, d, t, rb);
        }
    }
    if constexpr (C::KEPT) {
        F2 v[N2];
        post_vector(a.post_w, 1.0f, v);
        keep<N2, THREADS>(sgw, v);
        columns<VEC, NV, TPR>(a.w, 1.0f, d, t, v);
        keep<N2, THREADS>(sw, v);
        if constexpr (LAYER) {
            post_vector(a.post_b, 0.0f, v);
            keep<N2, THREADS>(sgb, v);
            columns<VEC, NV, TPR>(a.b, 0.0f, d, t, v);
            keep<N2, THREADS>(sb, v);
        }
    }
    for (; L::first(row) < a.R; row += step) {
        // y and the rest travel in groups of their own: each has a whole row's time
        cp_async_wait<1>();
        const bool there = row < a.R;
        const long long next = row + step;
        F2 v[N2];
        float ym = 0.0f, yr = 1.0f, xm = 0.0f, xr = 1.0f, shift = 0.0f;
        if (block) {
            F2 y[N2];
            fy.pairs(0, y);
            fy.issue(0, next, next < a.R);
            cp_async_commit();
            if (post) row_stats<VEC, NV, TPR, LAYER>(y, d, t, inv_d, a.eps, scratch, turn, ym, shift, yr);
            const F2 sh2 = f2(shift, shift), r2 = f2(yr, yr), al2 = f2(a.alpha, a.alpha);
            if constexpr (C::REGS) same<N2>(rgw, v);
            else if constexpr (C::KEPT) kept<N2, THREADS>(sgw, v);
            else post_vector(a.post_w, 1.0f, v);
            if constexpr (LAYER) {
                F2 b[N2];
                if constexpr (C::REGS) same<N2>(rgb, b);
                else if constexpr (C::KEPT) kept<N2, THREADS>(sgb, b);
                else post_vector(a.post_b, 0.0f, b);
#pragma unroll
                for (int k = 0; k < N2; ++k) y[k] = fma2(mul2(add2(y[k], sh2), r2), v[k], b[k]);
            } else {
#pragma unroll
                for (int k = 0; k < N2; ++k) y[k] = mul2(mul2(y[k], r2), v[k]);
            }
            cp_async_wait<1>();
            if (elem) {
                fg.pairs(0, v);
                fg.issue(0, next, next < a.R);
#pragma unroll
                for (int k = 0; k < N2; ++k) y[k] = mul2(y[k], v[k]);
            }
            fx.pairs(0, v);
#pragma unroll
            for (int k = 0; k < N2; ++k) v[k] = fma2(v[k], al2, y[k]);
            if (there) put<T, VEC, NV, TPR>(p.out + row * d, d, t, v);
        } else {
            cp_async_commit();
            cp_async_wait<1>();
            fx.pairs(0, v);
        }
        fx.issue(0, next, next < a.R);
        cp_async_commit();
        if (norm) {
            row_stats<VEC, NV, TPR, LAYER>(v, d, t, inv_d, a.eps, scratch, turn, xm, shift, xr);
            const F2 sh2 = f2(shift, shift), r2 = f2(xr, xr);
            F2 w[N2];
            if constexpr (C::REGS) same<N2>(rw, w);
            else if constexpr (C::KEPT) kept<N2, THREADS>(sw, w);
            else columns<VEC, NV, TPR>(a.w, 1.0f, d, t, w);
            if constexpr (LAYER) {
                F2 b[N2];
                if constexpr (C::REGS) same<N2>(rb, b);
                else if constexpr (C::KEPT) kept<N2, THREADS>(sb, b);
                else columns<VEC, NV, TPR>(a.b, 0.0f, d, t, b);
#pragma unroll
                for (int k = 0; k < N2; ++k) v[k] = fma2(mul2(add2(v[k], sh2), r2), w[k], b[k]);
            } else {
#pragma unroll
                for (int k = 0; k < N2; ++k) v[k] = mul2(mul2(v[k], r2), w[k]);
            }
            if (there) put<T, VEC, NV, TPR>(p.n + row * d, d, t, v);
        }
        if (t == 0 && there && a.stats != nullptr) {
            if constexpr (LAYER) {
                *stat(a, 0, static_cast<int>(row)) = ym;
                *stat(a, 2, static_cast<int>(row)) = xm;
            }
            *stat(a, 1, static_cast<int>(row)) = yr;
            *stat(a, 3, static_cast<int>(row)) = xr;
        }
    }
}

// Threads per row of the backward at width d, and CTAs of them on an SM.
// 16 columns a thread where the sums and what a row needs fit the registers: RMS of 16-bit types
// in vectors; else 8 (us, 16 : 8 columns, 100 to 200 MB: RMS, BF16, 8192 x 4096, 86 : 98, 65536 x 512,
// 69 : 89; layer, BF16, 8192 x 4096, 127 : 117, 65536 x 512, 109 : 102; layer, FP32, 8192 x 2048, 102 :
// 77). Single elements past 4096 columns: 1024 threads, else 16 columns.
enum BwdShape { BWD_SINGLE, BWD_8, BWD_16 };
constexpr int bwd_threads(int d, BwdShape shape) {
    if (shape != BWD_16)
        return d <= 8 * 8 ? 8 : d <= 32 * 8 ? 32 : d <= 64 * 8 ? 64 : d <= 96 * 8 ? 96 : d <= 128 * 8 ? 128 : d <= 192 * 8 ? 192 : d <= 256 * 8 ? 256 : d <= 512 * 8 || shape == BWD_8 ? 512 : 1024;
    return d <= 8 * 8 ? 8 : d <= 16 * 8 ? 16 : d <= 32 * 16 ? 32 : d <= 96 * 8 ? 96 : d <= 128 * 16 ? 128 : d <= 256 * 16 ? 256 : d <= 384 * 16 ? 384 : 512;
}
constexpr int bwd_per_sm(int tpr) { return tpr > 512 ? 1 : 512 / (tpr <= 32 ? 128 : tpr); }

template <typename T, int VEC, int NV, int TPR>
struct Backward {
    static constexpr int THREADS = RowThreads<TPR>::THREADS;
    using Fetch = Ahead<T, VEC, NV, TPR>;
    static constexpr int VECTOR = NV * VEC * 4 * THREADS;  // bytes of w, and of the gate times wp
    static constexpr int smem(int operands) { return 2 * VECTOR + operands * Fetch::SMEM; }
};

// A CTA walks rows and keeps its threads' columns of the sums in registers and of the vectors
// in shared memory (from L1, three of them a row: 8192 x 4096 BF16 86 us for 68);
// part[CTA] [RMS: S1, S3; layer: S1 .. S4][d] receives them.
template <typename T, int VEC, int NV, int TPR, bool LAYER>
__global__ void __launch_bounds__(Backward<T, VEC, NV, TPR>::THREADS, bwd_per_sm(TPR))
block_norm_bwd_kernel(const __grid_constant__ BlockNormArgs a, const __grid_constant__ Io<T> p, float* __restrict__ part) {
    using F = typename Backward<T, VEC, NV, TPR>::Fetch;
    using L = RowThreads<TPR>;
    constexpr int N2 = NV * VEC / 2, NS = LAYER ? 4 : 2;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float scratch[TPR > 32 ? 4 * (TPR / 32) : 1];
    __shared__ float gather[TPR <= 32 ? NV * VEC * TPR : 1];
    const int t = L::col(), d = a.d;
    const long long step = static_cast<long long>(gridDim.x) * L::ROWS;
    long long row = static_cast<long long>(blockIdx.x) * L::ROWS + L::row();
    const float inv_d = 1.0f / static_cast<float>(d);
    const bool block = p.y != nullptr, post = a.post != 0, norm = p.dn != nullptr, stream = p.dxo != nullptr, elem = p.g != nullptr;
    int turn = 0;
    F2 sum[NS][N2];  // RMS: S1, S3
#pragma unroll
    for (int q = 0; q < NS; ++q)
#pragma unroll
        for (int k = 0; k < N2; ++k) sum[q][k] = f2(0.0f, 0.0f);
    constexpr int S1 = 0, S2 = 1, S3 = NS / 2, S4 = NS - 1;
    pdl_wait();
    pdl_trigger();
    constexpr int THREADS = Backward<T, VEC, NV, TPR>::THREADS;
    F4* const sw = reinterpret_cast<F4*>(smem);
    F4* const sgw = sw + Backward<T, VEC, NV, TPR>::VECTOR / 16;
    uint8_t* const ahead = smem + 2 * Backward<T, VEC, NV, TPR>::VECTOR;
    F fx, fy, fn, fo, fg;
    fx.init(ahead, p.x, a.x_stride, d, t);
    fn.init(ahead + F::SMEM, p.dn, a.dn_stride, d, t);
    fo.init(ahead + 2 * F::SMEM, p.dxo, a.dxo_stride, d, t);
    fy.init(ahead + 3 * F::SMEM, p.y, a.y_stride, d, t);
    fg.init(ahead + 4 * F::SMEM, p.g, a.gate_stride, d, t);
    if (norm) {
        fx.issue(0, row, row < a.R);
        fn.issue(0, row, row < a.R);
    }
    cp_async_commit();
    if (stream) fo.issue(0, row, row < a.R);
    if (block) fy.issue(0, row, row < a.R);
    if (elem) fg.issue(0, row, row < a.R);
    cp_async_commit();
    {
        F2 w[N2], g[N2];
        columns<VEC, NV, TPR>(a.w, 1.0f, d, t, w);
        keep<N2, THREADS>(sw, w);
        columns<VEC, NV, TPR>(a.post_w, 1.0f, d, t, w);
        columns<VEC, NV, TPR>(a.gate, 1.0f, d, t, g);
#pragma unroll
        for (int k = 0; k < N2; ++k) w[k] = mul2(w[k], g[k]);
        keep<N2, THREADS>(sgw, w);
    }
    float ym = 0.0f, yr = 1.0f, xm = 0.0f, xr = 1.0f;  // of the next row
    auto statistics = [&](long long r) {
        if (r >= a.R) return;
        const int i = static_cast<int>(r);
        if (LAYER && post) ym = __ldg(stat(a, 0, i));
        if (post) yr = __ldg(stat(a, 1, i));
        if (LAYER && norm) xm = __ldg(stat(a, 2, i));
        if (norm) xr = __ldg(stat(a, 3, i));
    };
    statistics(row);
    for (; L::first(row) < a.R; row += step) {
        const bool there = row < a.R;
        const long long next = row + step;
        const bool more = next < a.R;
        cp_async_wait<1>();  // two groups a row, as in the forward
        const float ymc = ym, yrc = yr, xmc = xm, xrc = xr;
        statistics(row + step);
        F2 u[N2], v[N2];
        // of a warp whose other rows are there: shared memory holds an older row, or what was left there
        auto gone = [&](F2 (&q)[N2]) {
            if (TPR < 32 && !there) {
#pragma unroll
                for (int k = 0; k < N2; ++k) q[k] = f2(0.0f, 0.0f);
            }
        };
        // u: xh, v: h, then t
        if (norm) {
            fx.pairs(0, u);
            gone(u);
            fx.issue(0, next, more);
            fn.pairs(0, v);
            gone(v);
            fn.issue(0, next, more);
            cp_async_commit();
            const F2 r2 = f2(xrc, xrc);
            F2 a1 = f2(0.0f, 0.0f), a2 = a1;
            F2 w[N2];
            kept<N2, THREADS>(sw, w);
#pragma unroll
            for (int k = 0; k < N2; ++k) {
                // past the row's end dn is zero, and with it every term
                u[k] = mul2(LAYER ? less<VEC, TPR>(u[k], xmc, k, d, t) : u[k], r2);
                sum[S3][k] = fma2(v[k], u[k], sum[S3][k]);
                if constexpr (LAYER) sum[S4][k] = add2(sum[S4][k], v[k]);
                v[k] = mul2(v[k], w[k]);
                if constexpr (LAYER) a1 = add2(a1, v[k]);
                a2 = fma2(v[k], u[k], a2);
            }
            float s1 = both(a1), s2 = both(a2);
            if constexpr (LAYER) row_sum2<TPR>(s1, s2, scratch, turn);
            else row_sum<TPR>(s2, scratch, turn);
            s1 *= -inv_d;
            s2 *= -inv_d;
            const F2 n1 = f2(s1, s1), n2 = f2(s2, s2);
#pragma unroll
            for (int k = 0; k < N2; ++k) v[k] = mul2(fma2(u[k], n2, LAYER ? add2(v[k], n1) : v[k]), r2);
        } else {
            cp_async_commit();
        }
        cp_async_wait<1>();
        if (stream) {
            fo.pairs(0, u);
            gone(u);
            fo.issue(0, next, more);
#pragma unroll
            for (int k = 0; k < N2; ++k) v[k] = norm ? add2(v[k], u[k]) : u[k];
        }
        if (there) {
            const F2 al2 = f2(a.alpha, a.alpha);
#pragma unroll
            for (int k = 0; k < N2; ++k) u[k] = mul2(v[k], al2);
            put<T, VEC, NV, TPR>(p.out + row * d, d, t, u);
        }
        if (block) {
            // u: yh, v: t, t g, k, dy
            fy.pairs(0, u);
            gone(u);
            fy.issue(0, next, more);
            if (post) {
                const F2 r2 = f2(yrc, yrc);
#pragma unroll
                for (int k = 0; k < N2; ++k) u[k] = mul2(LAYER ? less<VEC, TPR>(u[k], ymc, k, d, t) : u[k], r2);
            }
            if (elem) {
                F2 z[N2];
                if (p.dgate != nullptr) {
                    F2 b[LAYER ? N2 : 1];
                    columns<VEC, NV, TPR>(a.post_w, 1.0f, d, t, z);
                    if constexpr (LAYER) columns<VEC, NV, TPR>(a.post_b, 0.0f, d, t, b);
#pragma unroll
                    for (int k = 0; k < N2; ++k) {
                        if constexpr (LAYER) z[k] = mul2(v[k], fma2(u[k], z[k], b[k]));
                        else z[k] = mul2(v[k], mul2(u[k], z[k]));
                    }
                    if (there) put<T, VEC, NV, TPR>(p.dgate + row * d, d, t, z);
                }
                fg.pairs(0, z);
                gone(z);
                fg.issue(0, next, more);
#pragma unroll
                for (int k = 0; k < N2; ++k) v[k] = mul2(v[k], z[k]);
            }
#pragma unroll
            for (int k = 0; k < N2; ++k) {
                sum[S1][k] = fma2(v[k], u[k], sum[S1][k]);
                if constexpr (LAYER) sum[S2][k] = add2(sum[S2][k], v[k]);
            }
            F2 wp[N2];  // the gate times wp: without a norm wp is 1
            kept<N2, THREADS>(sgw, wp);
            if (!post) {
#pragma unroll
                for (int k = 0; k < N2; ++k) v[k] = mul2(v[k], wp[k]);
            } else {
                F2 a1 = f2(0.0f, 0.0f), a2 = a1;
#pragma unroll
                for (int k = 0; k < N2; ++k) {
                    v[k] = mul2(v[k], wp[k]);  // zeros past the row's end
                    if constexpr (LAYER) a1 = add2(a1, v[k]);
                    a2 = fma2(v[k], u[k], a2);
                }
                float s1 = both(a1), s2 = both(a2);
                if constexpr (LAYER) row_sum2<TPR>(s1, s2, scratch, turn);
                else row_sum<TPR>(s2, scratch, turn);
                s1 *= -inv_d;
                s2 *= -inv_d;
                const F2 n1 = f2(s1, s1), n2 = f2(s2, s2), r2 = f2(yrc, yrc);
#pragma unroll
                for (int k = 0; k < N2; ++k) v[k] = mul2(fma2(u[k], n2, LAYER ? add2(v[k], n1) : v[k]), r2);
            }
            if (there) put<T, VEC, NV, TPR>(p.dy + row * d, d, t, v);
        }
        cp_async_commit();
    }
    if (part == nullptr) return;
    float* out = part + static_cast<long long>(blockIdx.x) * NS * d;
#pragma unroll
    for (int q = 0; q < NS; ++q) {
        float f[NV][VEC];
#pragma unroll
        for (int k = 0; k < N2; ++k) unpack(sum[q][k], f[2 * k / VEC][2 * k % VEC], f[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
        if constexpr (TPR <= 32) {
            // the CTA's rows in flight: one after the other into shared memory
            for (int w = 0; w < L::ROWS; ++w) {
                if (L::row() == w) {
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            const int at = (i * VEC + j) * TPR + t;
                            gather[at] = (w ? gather[at] : 0.0f) + f[i][j];
                        }
                }
                __syncthreads();
            }
            if (threadIdx.x < TPR) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int c = (i * TPR + t) * VEC + j;
                        if (c < d) out[q * d + c] = gather[(i * VEC + j) * TPR + t];
                    }
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * VEC;
                if (c < d) store_f32<VEC>(out + q * d + c, f[i]);
            }
        }
    }
}

constexpr int LONG_PARTS = 16;

bool vec_ok(const void* p, long long stride, int esz) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (stride * esz) % 16 == 0;
}
// Whether every operand's rows are on 16 bytes (all of them are read and written alike).
bool all_vec(const BlockNormArgs& a, int esz) {
    const long long d = a.d;
    return d * esz % 16 == 0 && vec_ok(a.x, a.x_stride, esz) && vec_ok(a.y, a.y_stride, esz) &&
           vec_ok(a.gate_elem, a.gate_stride, esz) && vec_ok(a.dn, a.dn_stride, esz) && vec_ok(a.dxo, a.dxo_stride, esz) &&
           vec_ok(a.out, 0, esz) && vec_ok(a.n, 0, esz) && vec_ok(a.dy, 0, esz) && vec_ok(a.dgate_elem, 0, esz) &&
           vec_ok(a.gate, 0, 4) && vec_ok(a.post_w, 0, 4) && vec_ok(a.post_b, 0, 4) && vec_ok(a.w, 0, 4) && vec_ok(a.b, 0, 4);
}

template <typename T, int VEC, int NV, int TPR, bool LAYER>
cudaError_t fwd_k(const BlockNormArgs& a, cudaStream_t s) {
    using C = Forward<T, VEC, NV, TPR, LAYER>;
    static bool done[64] = {};
    const int smem = C::smem(a.gate_elem != nullptr ? 3 : 2);
    if (!allow_smem(block_norm_kernel<T, VEC, NV, TPR, LAYER>, C::smem(3), done)) return cudaErrorInvalidValue;
    return launch_pdl(block_norm_kernel<T, VEC, NV, TPR, LAYER>, dim3(grid_rows(a.R, RowThreads<TPR>::ROWS, C::PER_SM)),
                      dim3(C::THREADS), smem, s, a, io_of<T>(a));
}

template <typename T, int VEC, bool LAYER>
cudaError_t fwd_v(const BlockNormArgs& a, cudaStream_t s) {
    const int d = a.d;
    if (d <= 8 * 8) return fwd_k<T, VEC, 8 / VEC, 8, LAYER>(a, s);
    if (d <= 32 * 8) return fwd_k<T, VEC, 8 / VEC, 32, LAYER>(a, s);
    if constexpr (VEC == 1) {  // 8 columns a thread: what a row needs, its vectors too, stays in registers
        if (d <= 64 * 8) return fwd_k<T, 1, 8, 64, LAYER>(a, s);
        if (d <= 128 * 8) return fwd_k<T, 1, 8, 128, LAYER>(a, s);
        if (d <= 192 * 8) return fwd_k<T, 1, 8, 192, LAYER>(a, s);
        if (d <= 256 * 8) return fwd_k<T, 1, 8, 256, LAYER>(a, s);
        if (d <= 512 * 8) return fwd_k<T, 1, 8, 512, LAYER>(a, s);
        if (d <= 1024 * 8) return fwd_k<T, 1, 8, 1024, LAYER>(a, s);
    } else {
        if (d <= 32 * 16) return fwd_k<T, VEC, 16 / VEC, 32, LAYER>(a, s);
        if (d <= 128 * 8) return fwd_k<T, VEC, 8 / VEC, 128, LAYER>(a, s);
        if (d <= 128 * 16) return fwd_k<T, VEC, 16 / VEC, 128, LAYER>(a, s);
        if (d <= 256 * 16) return fwd_k<T, VEC, 16 / VEC, 256, LAYER>(a, s);
        if (d <= 384 * 16) return fwd_k<T, VEC, 16 / VEC, 384, LAYER>(a, s);
        if (d <= 512 * 16) return fwd_k<T, VEC, 16 / VEC, 512, LAYER>(a, s);
    }
    return fwd_k<T, VEC, 16 / VEC, 1024, LAYER>(a, s);
}

template <typename T>
cudaError_t fwd_t(const BlockNormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (a.d > FWD_MAX_D)
        return launch_pdl(block_norm_long_kernel<T>, dim3(grid_rows(a.R, 1, 2)), dim3(LONG_THREADS), 0, s, a, io_of<T>(a));
    if (all_vec(a, sizeof(T))) return a.layer ? fwd_v<T, V, true>(a, s) : fwd_v<T, V, false>(a, s);
    return a.layer ? fwd_v<T, 1, true>(a, s) : fwd_v<T, 1, false>(a, s);
}

int bwd_parts(int R, int d, BwdShape shape) {
    if (d > BWD_MAX_D) return R < LONG_PARTS ? R : LONG_PARTS;
    const int t = bwd_threads(d, shape);
    return grid_rows(R, t <= 32 ? 128 / t : 1, bwd_per_sm(t));
}

template <typename T, int VEC, int NV, int TPR, bool LAYER>
cudaError_t bwd_k(const BlockNormArgs& a, int grid, float* part, cudaStream_t s) {
    using C = Backward<T, VEC, NV, TPR>;
    static bool done[64] = {};
    const int smem = C::smem(a.gate_elem != nullptr ? 5 : 4);
    if (!allow_smem(block_norm_bwd_kernel<T, VEC, NV, TPR, LAYER>, C::smem(5), done)) return cudaErrorInvalidValue;
    return launch_pdl(block_norm_bwd_kernel<T, VEC, NV, TPR, LAYER>, dim3(grid), dim3(C::THREADS), smem, s, a, io_of<T>(a), part);
}

template <typename T, int VEC, bool LAYER, BwdShape SHAPE>
cudaError_t bwd_v(const BlockNormArgs& a, float* part, cudaStream_t s) {
    const int n = bwd_parts(a.R, a.d, SHAPE);
    if constexpr (SHAPE == BWD_16) {
        switch (bwd_threads(a.d, SHAPE)) {
            case 8: return bwd_k<T, VEC, 8 / VEC, 8, LAYER>(a, n, part, s);
            case 16: return bwd_k<T, VEC, 8 / VEC, 16, LAYER>(a, n, part, s);
            case 32:
                if (a.d <= 32 * 8) return bwd_k<T, VEC, 8 / VEC, 32, LAYER>(a, n, part, s);
                return bwd_k<T, VEC, 16 / VEC, 32, LAYER>(a, n, part, s);
            case 96: return bwd_k<T, VEC, 8 / VEC, 96, LAYER>(a, n, part, s);
            case 128:
                if (a.d <= 128 * 8) return bwd_k<T, VEC, 8 / VEC, 128, LAYER>(a, n, part, s);
                return bwd_k<T, VEC, 16 / VEC, 128, LAYER>(a, n, part, s);
            case 256: return bwd_k<T, VEC, 16 / VEC, 256, LAYER>(a, n, part, s);
            case 384: return bwd_k<T, VEC, 16 / VEC, 384, LAYER>(a, n, part, s);
            default: return bwd_k<T, VEC, 16 / VEC, 512, LAYER>(a, n, part, s);
        }
    } else {
        switch (bwd_threads(a.d, SHAPE)) {
            case 8: return bwd_k<T, VEC, 8 / VEC, 8, LAYER>(a, n, part, s);
            case 32: return bwd_k<T, VEC, 8 / VEC, 32, LAYER>(a, n, part, s);
            case 64: return bwd_k<T, VEC, 8 / VEC, 64, LAYER>(a, n, part, s);
            case 96: return bwd_k<T, VEC, 8 / VEC, 96, LAYER>(a, n, part, s);
            case 128: return bwd_k<T, VEC, 8 / VEC, 128, LAYER>(a, n, part, s);
            case 192: return bwd_k<T, VEC, 8 / VEC, 192, LAYER>(a, n, part, s);
            case 256: return bwd_k<T, VEC, 8 / VEC, 256, LAYER>(a, n, part, s);
            case 512:
                if constexpr (SHAPE == BWD_8)
                    if (a.d > 512 * 8) return bwd_k<T, VEC, 16 / VEC, 512, LAYER>(a, n, part, s);
                return bwd_k<T, VEC, 8 / VEC, 512, LAYER>(a, n, part, s);
            default:
                if constexpr (SHAPE == BWD_SINGLE) return bwd_k<T, VEC, 8 / VEC, 1024, LAYER>(a, n, part, s);
                return cudaErrorInvalidValue;  // no such number of threads
        }
    }
}

template <typename T>
cudaError_t bwd_t(const BlockNormArgs& a, float* ws, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    constexpr BwdShape RMS = sizeof(T) == 2 ? BWD_16 : BWD_8;
    const bool vec = all_vec(a, sizeof(T));
    const int n = bwd_parts(a.R, a.d, !vec ? BWD_SINGLE : a.layer ? BWD_8 : RMS);
    cudaError_t e;
    if (a.d > BWD_MAX_D) {
        float* m12 = ws == nullptr ? nullptr : ws + static_cast<long long>(n) * (a.layer ? 4 : 2) * a.d;
        e = launch_pdl(block_norm_bwd_long_kernel<T>, dim3(grid_rows(a.R, 1, 2)), dim3(LONG_THREADS), 0, s, a, io_of<T>(a), m12);
        if (e == cudaSuccess && ws != nullptr)
            e = launch_pdl(block_norm_bwd_cols_kernel<T>, dim3((a.d + 255) / 256, n), dim3(256), 0, s, a, io_of<T>(a),
                           static_cast<const float*>(m12), ws);
    } else if (vec) {
        e = a.layer ? bwd_v<T, V, true, BWD_8>(a, ws, s) : bwd_v<T, V, false, RMS>(a, ws, s);
    } else {
        e = a.layer ? bwd_v<T, 1, true, BWD_SINGLE>(a, ws, s) : bwd_v<T, 1, false, BWD_SINGLE>(a, ws, s);
    }
    if (e != cudaSuccess || ws == nullptr) return e;
    return launch_block_norm_params(a, n, ws, s);
}

}  // namespace

}  // namespace moe
