// Layer norm in front of the layer, forward and backward.
//
//   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) rstd
//   y  = xh gamma + beta
//   g  = dy gamma;  dx = rstd (g - mean(g) - xh mean(g xh))
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Both are bound by memory: the forward reads x and writes y, the backward
// reads x and dy and writes dx, each element once. A row is held in registers
// by a warp (short rows) or by a CTA, 16 elements a thread, between its
// reduction and its output.
//
// Statistics are FP32. The forward sums the row, then the row less that mean:
// the second pass yields the squares and what rounding left in the mean, so a
// row whose mean is large against its deviation loses nothing.
#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

// Longest rows held in registers: 1024 threads x 16 elements; the backward,
// which keeps dgamma and dbeta besides, 512 x 16 (1024 threads leave 64
// registers each, and it spilled).
constexpr int FWD_MAX_D = 16384;
constexpr int BWD_MAX_D = 8192;

// 1 / sqrt(var + eps); a variance that rounding took below zero is zero, a NaN stays.
MOE_DEV float rstd_of(float var, float eps) { return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps); }

template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR)
layer_norm_kernel(int R, int d, const T* __restrict__ x, long long xs, const float* __restrict__ gamma,
                  const float* __restrict__ beta, float eps, T* __restrict__ y, long long ys,
                  float* __restrict__ mean, float* __restrict__ rstd) {
    constexpr int RPC = TPR == 32 ? 4 : 1;  // rows a CTA works on at a time
    __shared__ float scratch[TPR > 32 ? 4 * (TPR / 32) : 1];
    const int t = TPR == 32 ? static_cast<int>(lane_id()) : static_cast<int>(threadIdx.x);
    const long long step = static_cast<long long>(gridDim.x) * RPC;
    long long row = static_cast<long long>(blockIdx.x) * RPC + (TPR == 32 ? threadIdx.x >> 5 : 0);
    const float inv_d = 1.0f / static_cast<float>(d);
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    Raw<T, VEC> cur[NV];
    auto fetch = [&](long long r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (r < R && c < d)
                cur[i].load(x + r * xs + c);
            else
                cur[i].clear();
        }
    };
    fetch(row);
    for (; row < R; row += step) {
        float v[NV][VEC];
        float s = 0.0f, unused = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            cur[i].get(v[i]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) s += v[i][j];
        }
        fetch(row + step);  // the next row travels while this one is reduced
        row_sum2<TPR>(s, unused, scratch, turn);
        const float m0 = s * inv_d;
        float r1 = 0.0f, r2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = (i * TPR + t) * VEC < d;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                v[i][j] = in ? v[i][j] - m0 : 0.0f;
                r1 += v[i][j];
                r2 += v[i][j] * v[i][j];
            }
        }
        row_sum2<TPR>(r1, r2, scratch, turn);
        const float rest = r1 * inv_d;
        const float rs = rstd_of(r2 * inv_d - rest * rest, eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < d) {
                float o[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    o[j] = (v[i][j] - rest) * rs;
                    if (gamma != nullptr) o[j] *= __ldg(gamma + c + j);
                    if (beta != nullptr) o[j] += __ldg(beta + c + j);
                }
                Raw<T, VEC> out;
                out.set(o);
                out.store(y + row * ys + c);
            }
        }
        if (t == 0) {
            if (mean != nullptr) mean[row] = m0 + rest;
            if (rstd != nullptr) rstd[row] = rs;
        }
    }
}

// Rows longer than the registers hold: three passes, the later ones from L2.
template <typename T>
__global__ void __launch_bounds__(1024)
layer_norm_long_kernel(int R, int d, const T* __restrict__ x, long long xs, const float* __restrict__ gamma,
                       const float* __restrict__ beta, float eps, T* __restrict__ y, long long ys,
                       float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float scratch[4 * 32];
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    for (long long row = blockIdx.x; row < R; row += gridDim.x) {
        const T* xr = x + row * xs;
        float s = 0.0f, unused = 0.0f;
        for (int c = threadIdx.x; c < d; c += 1024) s += to_f32(xr[c]);
        row_sum2<1024>(s, unused, scratch, turn);
        const float m0 = s / static_cast<float>(d);
        float r1 = 0.0f, r2 = 0.0f;
        for (int c = threadIdx.x; c < d; c += 1024) {
            const float v = to_f32(xr[c]) - m0;
            r1 += v;
            r2 += v * v;
        }
        row_sum2<1024>(r1, r2, scratch, turn);
        const float rest = r1 / static_cast<float>(d);
        const float rs = rstd_of(r2 / static_cast<float>(d) - rest * rest, eps);
        for (int c = threadIdx.x; c < d; c += 1024) {
            float o = ((to_f32(xr[c]) - m0) - rest) * rs;
            if (gamma != nullptr) o *= gamma[c];
            if (beta != nullptr) o += beta[c];
            y[row * ys + c] = from_f32<T>(o);
        }
        if (threadIdx.x == 0) {
            if (mean != nullptr) mean[row] = m0 + rest;
            if (rstd != nullptr) rstd[row] = rs;
        }
    }
}

// Backward: a CTA walks rows and keeps its threads' columns of dgamma and
// dbeta in registers; part[cta] receives them, [2, d] FP32 each.
template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR)
layer_norm_bwd_kernel(int R, int d, const T* __restrict__ dy, long long dys, const T* __restrict__ x, long long xs,
                      const float* __restrict__ mean, const float* __restrict__ rstd,
                      const float* __restrict__ gamma, T* __restrict__ dx, long long dxs,
                      float* __restrict__ part) {
    constexpr int RPC = TPR == 32 ? 4 : 1;
    __shared__ float scratch[TPR > 32 ? 4 * (TPR / 32) : 1];
    __shared__ float gather[TPR == 32 ? 2 * NV * VEC * 32 : 1];
    const int t = TPR == 32 ? static_cast<int>(lane_id()) : static_cast<int>(threadIdx.x);
    const long long step = static_cast<long long>(gridDim.x) * RPC;
    long long row = static_cast<long long>(blockIdx.x) * RPC + (TPR == 32 ? threadIdx.x >> 5 : 0);
    const float inv_d = 1.0f / static_cast<float>(d);
    int turn = 0;
    float dg[NV][VEC] = {}, db[NV][VEC] = {};
    pdl_wait();
    pdl_trigger();
    Raw<T, VEC> cx[NV], cy[NV];
    auto fetch = [&](long long r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (r < R && c < d) {
                cx[i].load(x + r * xs + c);
                cy[i].load(dy + r * dys + c);
            } else {
                cx[i].clear();
                cy[i].clear();
            }
        }
    };
    fetch(row);
    for (; row < R; row += step) {
        const float mu = __ldg(mean + row), rs = __ldg(rstd + row);
        float xh[NV][VEC], g[NV][VEC];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            cx[i].get(xh[i]);
            cy[i].get(g[i]);
            if (c < d) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    xh[i][j] = (xh[i][j] - mu) * rs;
                    dg[i][j] += g[i][j] * xh[i][j];
                    db[i][j] += g[i][j];
                    if (gamma != nullptr) g[i][j] *= __ldg(gamma + c + j);
                    s1 += g[i][j];
                    s2 += g[i][j] * xh[i][j];
                }
            }
        }
        fetch(row + step);
        row_sum2<TPR>(s1, s2, scratch, turn);
        s1 *= inv_d;
        s2 *= inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < d) {
                float o[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) o[j] = rs * (g[i][j] - s1 - xh[i][j] * s2);
                Raw<T, VEC> out;
                out.set(o);
                out.store(dx + row * dxs + c);
            }
        }
    }
    if (part == nullptr) return;
    float* pg = part + static_cast<long long>(blockIdx.x) * 2 * d;
    if constexpr (TPR == 32) {
        // the CTA's four rows in flight: one after the other into shared memory
        constexpr int N = NV * VEC;
        for (int w = 0; w < RPC; ++w) {
            if (static_cast<int>(threadIdx.x >> 5) == w) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int a = (i * VEC + j) * 32 + t;
                        gather[a] = (w ? gather[a] : 0.0f) + dg[i][j];
                        gather[N * 32 + a] = (w ? gather[N * 32 + a] : 0.0f) + db[i][j];
                    }
            }
            __syncthreads();
        }
        if (threadIdx.x < 32) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int c = (i * 32 + t) * VEC + j, a = (i * VEC + j) * 32 + t;
                    if (c < d) {
                        pg[c] = gather[a];
                        pg[d + c] = gather[N * 32 + a];
                    }
                }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int c = (i * TPR + t) * VEC + j;
                if (c < d) {
                    pg[c] = dg[i][j];
                    pg[d + c] = db[i][j];
                }
            }
    }
}

// Longer rows: the row's sums, then dx; the columns' sums by their own kernel.
template <typename T>
__global__ void __launch_bounds__(1024)
layer_norm_bwd_long_kernel(int R, int d, const T* __restrict__ dy, long long dys, const T* __restrict__ x,
                           long long xs, const float* __restrict__ mean, const float* __restrict__ rstd,
                           const float* __restrict__ gamma, T* __restrict__ dx, long long dxs) {
    __shared__ float scratch[4 * 32];
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    for (long long row = blockIdx.x; row < R; row += gridDim.x) {
        const float mu = mean[row], rs = rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < d; c += 1024) {
            const float g = to_f32(dy[row * dys + c]) * (gamma != nullptr ? gamma[c] : 1.0f);
            s1 += g;
            s2 += g * ((to_f32(x[row * xs + c]) - mu) * rs);
        }
        row_sum2<1024>(s1, s2, scratch, turn);
        s1 /= static_cast<float>(d);
        s2 /= static_cast<float>(d);
        for (int c = threadIdx.x; c < d; c += 1024) {
            const float g = to_f32(dy[row * dys + c]) * (gamma != nullptr ? gamma[c] : 1.0f);
            dx[row * dxs + c] = from_f32<T>(rs * (g - s1 - (to_f32(x[row * xs + c]) - mu) * rs * s2));
        }
    }
}
template <typename T>
__global__ void __launch_bounds__(256)
layer_norm_bwd_cols_kernel(int R, int d, const T* __restrict__ dy, long long dys, const T* __restrict__ x,
                           long long xs, const float* __restrict__ mean, const float* __restrict__ rstd,
                           float* __restrict__ part) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (c >= d) return;
    float dg = 0.0f, db = 0.0f;
    for (long long r = blockIdx.y; r < R; r += gridDim.y) {
        const float g = to_f32(dy[r * dys + c]);
        dg += g * ((to_f32(x[r * xs + c]) - mean[r]) * rstd[r]);
        db += g;
    }
    part[static_cast<long long>(blockIdx.y) * 2 * d + c] = dg;
    part[static_cast<long long>(blockIdx.y) * 2 * d + d + c] = db;
}

// dgamma, dbeta = the sums of the n partial rows [2, d], each column in a
// fixed order: 8 threads take every eighth row, then add theirs in order.
__global__ void __launch_bounds__(256)
layer_norm_cols_sum_kernel(int n, int d, const float* __restrict__ part, float* __restrict__ dgamma,
                           float* __restrict__ dbeta) {
    __shared__ float s[8][32];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    pdl_wait();
    pdl_trigger();
    float a = 0.0f;
    if (c < 2 * d) {
        int r = ry;
        for (; r + 24 < n; r += 32) {  // four loads in flight
            const float p0 = part[static_cast<long long>(r) * 2 * d + c];
            const float p1 = part[static_cast<long long>(r + 8) * 2 * d + c];
            const float p2 = part[static_cast<long long>(r + 16) * 2 * d + c];
            const float p3 = part[static_cast<long long>(r + 24) * 2 * d + c];
            a += (p0 + p1) + (p2 + p3);
        }
        for (; r < n; r += 8) a += part[static_cast<long long>(r) * 2 * d + c];
    }
    s[ry][cx] = a;
    __syncthreads();
    if (ry == 0 && c < 2 * d) {
        float v = s[0][cx];
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][cx];
        if (c < d) {
            if (dgamma != nullptr) dgamma[c] = v;
        } else if (dbeta != nullptr) {
            dbeta[c - d] = v;
        }
    }
}

bool vec_ok(const void* p, long long stride, int esz) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (stride * esz) % 16 == 0;
}

int grid_rows(long long rows, int rpc, int per_sm) {
    const long long want = (rows + rpc - 1) / rpc, cap = static_cast<long long>(num_sms()) * per_sm;
    return static_cast<int>(want < cap ? want : cap);
}

// CTAs of the backward, and so partial rows of its workspace.
constexpr int BWD_PER_SM = 2;

template <typename T, int VEC, int NV, int TPR>
cudaError_t fwd_t(const LayerNormArgs& a, cudaStream_t s) {
    const int rpc = TPR == 32 ? 4 : 1, threads = TPR == 32 ? 128 : TPR;
    const int grid = grid_rows(a.R, rpc, 2048 / threads);
    return launch_pdl(layer_norm_kernel<T, VEC, NV, TPR>, dim3(grid), dim3(threads), 0, s, a.R, a.d,
                      static_cast<const T*>(a.x), a.x_stride, a.gamma, a.beta, a.eps, static_cast<T*>(a.y),
                      a.y_stride, a.mean_out, a.rstd_out);
}

template <typename T, int VEC>
cudaError_t fwd_v(const LayerNormArgs& a, cudaStream_t s) {
    const int d = a.d;
    if (d <= 32 * 8) return fwd_t<T, VEC, 8 / VEC, 32>(a, s);
    if (d <= 32 * 32) return fwd_t<T, VEC, 32 / VEC, 32>(a, s);
    if (d <= 128 * 16) return fwd_t<T, VEC, 16 / VEC, 128>(a, s);
    if (d <= 256 * 16) return fwd_t<T, VEC, 16 / VEC, 256>(a, s);
    return fwd_t<T, VEC, 16 / VEC, 1024>(a, s);
}

template <typename T>
cudaError_t fwd_d(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (a.d > FWD_MAX_D)
        return launch_pdl(layer_norm_long_kernel<T>, dim3(grid_rows(a.R, 1, 2)), dim3(1024), 0, s, a.R, a.d,
                          static_cast<const T*>(a.x), a.x_stride, a.gamma, a.beta, a.eps, static_cast<T*>(a.y),
                          a.y_stride, a.mean_out, a.rstd_out);
    if (a.d % V == 0 && vec_ok(a.x, a.x_stride, sizeof(T)) && vec_ok(a.y, a.y_stride, sizeof(T)))
        return fwd_v<T, V>(a, s);
    return fwd_v<T, 1>(a, s);
}

template <typename T, int VEC, int NV, int TPR>
cudaError_t bwd_t(const LayerNormArgs& a, int grid, float* part, cudaStream_t s) {
    const int threads = TPR == 32 ? 128 : TPR;
    return launch_pdl(layer_norm_bwd_kernel<T, VEC, NV, TPR>, dim3(grid), dim3(threads), 0, s, a.R, a.d,
                      static_cast<const T*>(a.dy), a.dy_stride, static_cast<const T*>(a.x), a.x_stride, a.mean,
                      a.rstd, a.gamma, static_cast<T*>(a.y), a.y_stride, part);
}

template <typename T, int VEC>
cudaError_t bwd_v(const LayerNormArgs& a, int grid, float* part, cudaStream_t s) {
    const int d = a.d;
    if (d <= 32 * 8) return bwd_t<T, VEC, 8 / VEC, 32>(a, grid, part, s);
    if (d <= 128 * 8) return bwd_t<T, VEC, 8 / VEC, 128>(a, grid, part, s);
    if (d <= 256 * 16) return bwd_t<T, VEC, 16 / VEC, 256>(a, grid, part, s);
    return bwd_t<T, VEC, 16 / VEC, 512>(a, grid, part, s);
}

template <typename T>
cudaError_t bwd_d(const LayerNormArgs& a, float* part, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    int n = layer_norm_bwd_parts(a.R, a.d);
    cudaError_t e;
    if (a.d > BWD_MAX_D) {
        e = launch_pdl(layer_norm_bwd_long_kernel<T>, dim3(grid_rows(a.R, 1, 2)), dim3(1024), 0, s, a.R, a.d,
                       static_cast<const T*>(a.dy), a.dy_stride, static_cast<const T*>(a.x), a.x_stride, a.mean,
                       a.rstd, a.gamma, static_cast<T*>(a.y), a.y_stride);
        if (e == cudaSuccess && part != nullptr)
            e = launch_pdl(layer_norm_bwd_cols_kernel<T>, dim3((a.d + 255) / 256, n), dim3(256), 0, s, a.R, a.d,
                           static_cast<const T*>(a.dy), a.dy_stride, static_cast<const T*>(a.x), a.x_stride,
                           a.mean, a.rstd, part);
    } else if (a.d % V == 0 && vec_ok(a.x, a.x_stride, sizeof(T)) && vec_ok(a.dy, a.dy_stride, sizeof(T)) &&
               vec_ok(a.y, a.y_stride, sizeof(T))) {
        e = bwd_v<T, V>(a, n, part, s);
    } else {
        e = bwd_v<T, 1>(a, n, part, s);
    }
    if (e != cudaSuccess || part == nullptr) return e;
    return launch_pdl(layer_norm_cols_sum_kernel, dim3((2 * a.d + 31) / 32), dim3(256), 0, s, n, a.d,
                      static_cast<const float*>(part), a.dgamma, a.dbeta);
}

}  // namespace

int layer_norm_bwd_parts(int R, int d) {
    if (d > BWD_MAX_D) return R < 16 ? R : 16;
    return grid_rows(R, d <= 256 ? 4 : 1, BWD_PER_SM);
}

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s) {
    switch (a.dtype) {
        case MOE_BF16: return fwd_d<__nv_bfloat16>(a, s);
        case MOE_F16: return fwd_d<__half>(a, s);
        default: return fwd_d<float>(a, s);
    }
}

cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, float* part, cudaStream_t s) {
    switch (a.dtype) {
        case MOE_BF16: return bwd_d<__nv_bfloat16>(a, part, s);
        case MOE_F16: return bwd_d<__half>(a, part, s);
        default: return bwd_d<float>(a, part, s);
    }
}

}  // namespace moe
