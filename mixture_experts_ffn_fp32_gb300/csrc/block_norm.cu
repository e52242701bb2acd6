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

MOE_DEV float rstd_of(float var, float eps) { return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps); }

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
    mean = m0 + rest;
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

template <typename T>
cudaError_t fwd_t(const BlockNormArgs& a, cudaStream_t s) {
    return launch_pdl(block_norm_long_kernel<T>, dim3(grid_rows(a.R, 1, 2)), dim3(LONG_THREADS), 0, s, a, io_of<T>(a));
}

constexpr int LONG_PARTS = 16;

template <typename T>
cudaError_t bwd_t(const BlockNormArgs& a, float* ws, cudaStream_t s) {
    const int n = a.R < LONG_PARTS ? a.R : LONG_PARTS;
    float* part = ws;
    float* m12 = ws == nullptr ? nullptr : ws + static_cast<long long>(n) * (a.layer ? 4 : 2) * a.d;
    cudaError_t e = launch_pdl(block_norm_bwd_long_kernel<T>, dim3(grid_rows(a.R, 1, 2)), dim3(LONG_THREADS), 0, s, a,
                               io_of<T>(a), m12);
    if (e == cudaSuccess && ws != nullptr)
        e = launch_pdl(block_norm_bwd_cols_kernel<T>, dim3((a.d + 255) / 256, n), dim3(256), 0, s, a, io_of<T>(a),
                       static_cast<const float*>(m12), part);
    if (e != cudaSuccess || ws == nullptr) return e;
    const dim3 grid((a.d + 31) / 32), block(32 * COL_ROWS);
    return a.layer ? launch_pdl(block_norm_params_kernel<4>, grid, block, 0, s, a, n, static_cast<const float*>(part))
                   : launch_pdl(block_norm_params_kernel<2>, grid, block, 0, s, a, n, static_cast<const float*>(part));
}

}  // namespace

size_t block_norm_bwd_floats(int R, int d, bool layer) {
    const size_t n = R < LONG_PARTS ? R : LONG_PARTS;
    return n * (layer ? 4 : 2) * d + 2 * static_cast<size_t>(R);
}

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s) {
    switch (a.dtype) {
        case MOE_BF16: return fwd_t<__nv_bfloat16>(a, s);
        case MOE_F16: return fwd_t<__half>(a, s);
        default: return fwd_t<float>(a, s);
    }
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, float* ws, cudaStream_t s) {
    switch (a.dtype) {
        case MOE_BF16: return bwd_t<__nv_bfloat16>(a, ws, s);
        case MOE_F16: return bwd_t<__half>(a, ws, s);
        default: return bwd_t<float>(a, ws, s);
    }
}

}  // namespace moe
