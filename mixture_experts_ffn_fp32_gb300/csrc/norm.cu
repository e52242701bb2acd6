// Layer norm in front of the layer, forward and backward.
//
//   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) rstd
//   y  = xh gamma + beta
//   g  = dy gamma;  dx = rstd (g - mean(g) - xh mean(g xh))
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Both are bound by memory: the forward reads x and writes y, the backward
// reads x and dy and writes dx, each element once. A row is held in registers
// by part of a warp (short rows) or by a CTA, up to 16 elements a thread (32 where
// a warp holds a row of up to 1024 in the forward), between its reduction and its
// output, while the next rows of the CTA travel into shared memory.
//
// Statistics are FP32. The forward sums the row, then the row less a mean: the
// second sums yield the squares and what rounding left in the mean, so a row
// whose mean is large against its deviation loses nothing.
//
// Measured (one GB300, 6.8 TB/s copy rate, caches cold): forward, 16384 x 2048
// BF16 26 us (5.2 TB/s), 8192 x 4096 FP32 5.5 TB/s; backward, 8192 x 4096 BF16
// 33 us and 5 for the column sums (6.1 TB/s; 41 before the CTAs' partial sums
// were stored 16 bytes at a time), 5003 x 1411 FP32 unaligned 19 + 5 us. BF16
// rows are held back by instructions and their latencies: 1200 a row of 2048 forward
// keep 65 % of the issue slots busy and 2290 a row of 4096 backward 50 %, and the
// commonest waits are for shuffles and shared memory. Packed FP32 pairs took 29 us to
// 26 forward and 45 to 41 backward; more rows ahead or more CTAs do not help (35 us with
// 1216 CTAs, each of which reads gamma and beta again). Few rows are latency: 128 x 4096
// 4 us. Rows that registers do not hold are read two or three times, element by element:
// 4096 x 20480 BF16 forward 136 us (2.5 TB/s), 8192 x 12288 backward 363 us (1.7 TB/s).
#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

// Longest rows held in registers: 1024 threads x 16 elements; the backward,
// which keeps dgamma and dbeta besides, 512 x 16 (1024 threads leave 64
// registers each, and it spilled).
constexpr int FWD_MAX_D = 16384;
constexpr int BWD_MAX_D = 8192;
// Rows that travel ahead of the one a CTA works on.
constexpr int FWD_DEPTH = 3;
constexpr int BWD_DEPTH = 2;

// 1 / sqrt(var + eps); a variance that rounding took below zero is zero, a NaN stays.
MOE_DEV float rstd_of(float var, float eps) { return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps); }

// A mean and what rounding left in it, which is no number where the mean is infinite.
MOE_DEV float joined(float m, float rest) { return rest == rest ? m + rest : m; }

// Mean and variance of a row from its threads' NV x VEC values (in pairs), left
// as v - m, m a mean the warp took of its own. Its sums of the differences and of
// their squares follow, and the CTA joins the warps' numbers (m, r, q of n values)
// behind one sync:
//   m0 = sum n m / d,  rest = sum (n (m - m0) + r) / d
//   var = sum (q + 2 (m - m0) r + n (m - m0)^2) / d - rest^2
// `rest` is what rounding left in m0; shift = m - (m0 + rest).
template <int VEC, int NV, int TPR>
MOE_DEV void row_moments(F2 (&v)[NV * VEC / 2], int d, int t, float inv_d, float4* scratch, int& turn, float& mean,
                         float& shift, float& var) {
    constexpr int W = TPR <= 32 ? 1 : TPR / 32, N2 = NV * VEC / 2;
    const int w = W == 1 ? 0 : static_cast<int>(threadIdx.x >> 5);
    constexpr int S = TPR < 32 ? TPR : 32;  // threads that sum by shuffles
    float n = 0.0f;  // the warp's values, cut at d
#pragma unroll
    for (int i = 0; i < NV; ++i) n += static_cast<float>(min(max(d - (i * TPR + w * 32) * VEC, 0), S * VEC));
    F2 s2 = v[0];
#pragma unroll
    for (int k = 1; k < N2; ++k) s2 = add2(s2, v[k]);
    const float s = seg_sum<S>(both(s2));
    const float m = W == 1 ? s * inv_d : (n > 0.0f ? s / n : 0.0f);
    F2 r2 = f2(0.0f, 0.0f), q2 = r2;
#pragma unroll
    for (int k = 0; k < N2; ++k) {
        // zeros past the end stay zeros
        const float ma = (2 * k / VEC * TPR + t) * VEC < d ? -m : 0.0f;
        const float mb = VEC > 1 ? ma : ((2 * k + 1) * TPR + t < d ? -m : 0.0f);
        v[k] = add2(v[k], f2(ma, mb));
        r2 = add2(r2, v[k]);
        q2 = fma2(v[k], v[k], q2);
    }
    const float r = seg_sum<S>(both(r2)), q = seg_sum<S>(both(q2));
    if constexpr (W == 1) {
        const float rest = r * inv_d;
        mean = joined(m, rest);
        shift = -rest;
        var = q * inv_d - rest * rest;
    } else {
        float4* sc = scratch + (turn & 1) * W;  // two turns: see row_sum2
        ++turn;
        if (lane_id() == 0) sc[w] = make_float4(m, r, q, n);
        __syncthreads();
        const int l = static_cast<int>(lane_id());
        float4 e = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (l < W) e = sc[l];
        const float m0 = group_sum<W>(e.w * e.x) * inv_d;
        const float dm = e.x - m0;
        const float rest = group_sum<W>(e.w * dm + e.y) * inv_d;
        var = group_sum<W>(e.z + 2.0f * dm * e.y + e.w * dm * dm) * inv_d - rest * rest;
        mean = joined(m0, rest);
        shift = (m - m0) - rest;
    }
}

template <typename T, int VEC, int NV, int TPR>
struct Forward {
    static constexpr int THREADS = RowThreads<TPR>::THREADS;
    // CTAs of an SM: as many threads as the registers of a thread's columns leave
    static constexpr int PER_SM = (TPR == 1024 ? 1024
                                   : NV * VEC <= 4 ? 1536
                                   : NV * VEC <= 8 ? 1024
                                   : VEC == 1 || TPR == 512 || NV * VEC > 16 ? 512
                                                                            : 768) / THREADS;
    // gamma and beta stay in registers where a thread has few columns
    static constexpr bool KEEP = VEC > 1 && NV * VEC <= 16 && TPR < 1024;
    using Fetch = RowFetch<T, VEC, NV, TPR, THREADS, FWD_DEPTH>;
};

template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(Forward<T, VEC, NV, TPR>::THREADS, Forward<T, VEC, NV, TPR>::PER_SM)
layer_norm_kernel(int R, int d, const T* __restrict__ x, long long xs, const float* __restrict__ gamma,
                  const float* __restrict__ beta, float eps, T* __restrict__ y, long long ys,
                  float* __restrict__ mean, float* __restrict__ rstd) {
    using F = typename Forward<T, VEC, NV, TPR>::Fetch;
    constexpr int D = F::D;
    using L = RowThreads<TPR>;
    constexpr bool KEEP = Forward<T, VEC, NV, TPR>::KEEP;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float4 scratch[TPR > 32 ? 2 * (TPR / 32) : 1];
    const int t = L::col();
    const long long step = static_cast<long long>(gridDim.x) * L::ROWS;
    long long row = static_cast<long long>(blockIdx.x) * L::ROWS + L::row();
    const float inv_d = 1.0f / static_cast<float>(d);
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    F in;
    in.init(smem, x, xs, d, t);
#pragma unroll
    for (int s = 0; s < D; ++s) {
        in.issue(s, row + s * step, row + s * step < R);
        if constexpr (F::ASYNC) cp_async_commit();
    }
    constexpr int N2 = NV * VEC / 2;
    F2 ga[N2], be[N2];
    auto columns = [&] {
        float g[NV][VEC], b[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                g[i][j] = 1.0f;
                b[i][j] = 0.0f;
            }
            if (c < d && gamma != nullptr) load_f32<VEC>(gamma + c, g[i]);
            if (c < d && beta != nullptr) load_f32<VEC>(beta + c, b[i]);
        }
#pragma unroll
        for (int k = 0; k < N2; ++k) {
            constexpr int V = VEC;
            ga[k] = f2(g[2 * k / V][2 * k % V], g[(2 * k + 1) / V][(2 * k + 1) % V]);
            be[k] = f2(b[2 * k / V][2 * k % V], b[(2 * k + 1) / V][(2 * k + 1) % V]);
        }
    };
    if constexpr (KEEP) columns();
    int slot = 0;
    for (; L::first(row) < R; row += step) {
        F2 v[N2];
        if constexpr (F::ASYNC) cp_async_wait<D - 1>();
        in.pairs(slot, v);
        in.issue(slot, row + D * step, row + D * step < R);
        if constexpr (F::ASYNC) cp_async_commit();
        if (++slot == D) slot = 0;
        float m, shift, var;
        row_moments<VEC, NV, TPR>(v, d, t, inv_d, scratch, turn, m, shift, var);
        const float rs = rstd_of(var, eps);
        if constexpr (!KEEP) columns();
        const F2 sh2 = f2(shift, shift), rs2 = f2(rs, rs);
        float o[NV][VEC];
#pragma unroll
        for (int k = 0; k < N2; ++k) {
            const F2 y2 = fma2(mul2(add2(v[k], sh2), rs2), ga[k], be[k]);
            unpack(y2, o[2 * k / VEC][2 * k % VEC], o[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < d && row < R) {
                Raw<T, VEC> out;
                out.set(o[i]);
                out.store(y + row * ys + c);
            }
        }
        if (t == 0 && row < R) {
            if (mean != nullptr) mean[row] = m;
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
            if (mean != nullptr) mean[row] = joined(m0, rest);
            if (rstd != nullptr) rstd[row] = rs;
        }
    }
}

// Threads per row of the backward at width d, and CTAs of them on an SM. (16
// threads for rows to 128, 32 of 16 columns to 512: 100000 BF16 rows of 128 39 -> 29 us,
// 34605 of 320 43 -> 25. 192 and 384 leave fewer threads without columns; BF16 rows of
// 2560, 5120, 100 MB: 70 -> 66, 74 -> 70 us. 96 gained nothing, and three CTAs of 192
// spilled: 96 us.)
constexpr int bwd_threads(int d) {
    return d <= 8 * 8 ? 8 : d <= 16 * 8 ? 16 : d <= 32 * 16 ? 32 : d <= 128 * 16 ? 128 : d <= 192 * 16 ? 192 : d <= 256 * 16 ? 256 : d <= 384 * 16 ? 384 : 512;
}
constexpr int bwd_per_sm(int tpr) { return 512 / (tpr <= 32 ? 128 : tpr); }

template <typename T, int VEC, int NV, int TPR>
struct Backward {
    static constexpr int THREADS = RowThreads<TPR>::THREADS;
    using Fetch = RowFetch<T, VEC, NV, TPR, THREADS, BWD_DEPTH>;
};

// Backward: a CTA walks rows and keeps its threads' columns of dgamma and
// dbeta in registers; part[cta] receives them, [2, d] FP32 each.
template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(Backward<T, VEC, NV, TPR>::THREADS, bwd_per_sm(TPR))
layer_norm_bwd_kernel(int R, int d, const T* __restrict__ dy, long long dys, const T* __restrict__ x, long long xs,
                      const float* __restrict__ mean, const float* __restrict__ rstd,
                      const float* __restrict__ gamma, T* __restrict__ dx, long long dxs,
                      float* __restrict__ part) {
    using F = typename Backward<T, VEC, NV, TPR>::Fetch;
    constexpr int D = F::D;
    using L = RowThreads<TPR>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float scratch[TPR > 32 ? 4 * (TPR / 32) : 1];
    __shared__ float gather[TPR <= 32 ? 2 * NV * VEC * TPR : 1];
    const int t = L::col();
    const long long step = static_cast<long long>(gridDim.x) * L::ROWS;
    long long row = static_cast<long long>(blockIdx.x) * L::ROWS + L::row();
    const float inv_d = 1.0f / static_cast<float>(d);
    int turn = 0;
    constexpr int N2 = NV * VEC / 2;
    constexpr bool KEEP = VEC > 1;  // gamma in registers
    F2 dg2[N2], db2[N2], ga[N2];
#pragma unroll
    for (int k = 0; k < N2; ++k) dg2[k] = db2[k] = f2(0.0f, 0.0f);
    pdl_wait();
    pdl_trigger();
    F fx, fy;
    fx.init(smem, x, xs, d, t);
    fy.init(smem + F::SMEM, dy, dys, d, t);
    auto issue = [&](int s, long long r) {
        fx.issue(s, r, r < R);
        fy.issue(s, r, r < R);
        if constexpr (F::ASYNC) cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < D; ++s) issue(s, row + s * step);
    auto columns = [&] {
        float g[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) g[i][j] = 1.0f;
            if (c < d && gamma != nullptr) load_f32<VEC>(gamma + c, g[i]);
        }
#pragma unroll
        for (int k = 0; k < N2; ++k) ga[k] = f2(g[2 * k / VEC][2 * k % VEC], g[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
    };
    if constexpr (KEEP) columns();
    float mu = 0.0f, rs = 0.0f;  // of the next row
    if (row < R) {
        mu = __ldg(mean + row);
        rs = __ldg(rstd + row);
    }
    int slot = 0;
    for (; L::first(row) < R; row += step) {
        F2 xh[N2], g[N2];
        const float mc = mu, rc = rs;
        if (row + step < R) {
            mu = __ldg(mean + row + step);
            rs = __ldg(rstd + row + step);
        }
        if constexpr (F::ASYNC) cp_async_wait<D - 1>();
        fx.pairs(slot, xh);
        fy.pairs(slot, g);
        if (TPR < 32 && row >= R) {  // of a warp whose other rows are there
#pragma unroll
            for (int k = 0; k < N2; ++k) xh[k] = g[k] = f2(0.0f, 0.0f);
        }
        issue(slot, row + D * step);
        if (++slot == D) slot = 0;
        if constexpr (!KEEP) columns();
        const F2 nm = f2(-mc, -mc), rc2 = f2(rc, rc);
        F2 a1 = f2(0.0f, 0.0f), a2 = a1;
#pragma unroll
        for (int k = 0; k < N2; ++k) {
            // past the row's end dy is zero, and with it every term
            xh[k] = mul2(add2(xh[k], nm), rc2);
            dg2[k] = fma2(g[k], xh[k], dg2[k]);
            db2[k] = add2(db2[k], g[k]);
            g[k] = mul2(g[k], ga[k]);
            a1 = add2(a1, g[k]);
            a2 = fma2(g[k], xh[k], a2);
        }
        float s1 = both(a1), s2 = both(a2);
        row_sum2<TPR>(s1, s2, scratch, turn);
        s1 *= -inv_d;
        s2 *= -inv_d;
        const F2 n1 = f2(s1, s1), n2 = f2(s2, s2);
        float o[NV][VEC];
#pragma unroll
        for (int k = 0; k < N2; ++k) {
            const F2 x2 = mul2(fma2(xh[k], n2, add2(g[k], n1)), rc2);
            unpack(x2, o[2 * k / VEC][2 * k % VEC], o[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < d && row < R) {
                Raw<T, VEC> out;
                out.set(o[i]);
                out.store(dx + row * dxs + c);
            }
        }
    }
    float dg[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int k = 0; k < N2; ++k) {
        unpack(dg2[k], dg[2 * k / VEC][2 * k % VEC], dg[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
        unpack(db2[k], db[2 * k / VEC][2 * k % VEC], db[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
    }
    if (part == nullptr) return;
    float* pg = part + static_cast<long long>(blockIdx.x) * 2 * d;
    if constexpr (TPR <= 32) {
        // the CTA's rows in flight: one after the other into shared memory
        constexpr int N = NV * VEC;
        for (int w = 0; w < L::ROWS; ++w) {
            if (L::row() == w) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int a = (i * VEC + j) * TPR + t;
                        gather[a] = (w ? gather[a] : 0.0f) + dg[i][j];
                        gather[N * TPR + a] = (w ? gather[N * TPR + a] : 0.0f) + db[i][j];
                    }
            }
            __syncthreads();
        }
        if (threadIdx.x < TPR) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int c = (i * TPR + t) * VEC + j, a = (i * VEC + j) * TPR + t;
                    if (c < d) {
                        pg[c] = gather[a];
                        pg[d + c] = gather[N * TPR + a];
                    }
                }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < d) {  // 16-byte stores (4-byte ones, a sector each: 41 us for 33)
                store_f32<VEC>(pg + c, dg[i]);
                store_f32<VEC>(pg + d + c, db[i]);
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
// fixed order: 32 threads take every 32nd row, ten loads in flight (the rows
// of two CTAs an SM in one go), then theirs are added in order.
constexpr int COL_ROWS = 32;
__global__ void __launch_bounds__(32 * COL_ROWS)
layer_norm_cols_sum_kernel(int n, int d, const float* __restrict__ part, float* __restrict__ dgamma,
                           float* __restrict__ dbeta) {
    __shared__ float s[COL_ROWS][32];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    pdl_wait();
    pdl_trigger();
    float a = 0.0f;
    if (c < 2 * d) {
        for (int r0 = ry; r0 < n; r0 += 10 * COL_ROWS) {
            float p[10];
#pragma unroll
            for (int i = 0; i < 10; ++i) {
                const int r = r0 + i * COL_ROWS;
                p[i] = r < n ? part[static_cast<long long>(r) * 2 * d + c] : 0.0f;
            }
            a += (((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]))) + (p[8] + p[9]);
        }
    }
    s[ry][cx] = a;
    __syncthreads();
    if (ry == 0 && c < 2 * d) {
        float v = s[0][cx];
#pragma unroll
        for (int i = 1; i < COL_ROWS; ++i) v += s[i][cx];
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

template <typename T, int VEC, int NV, int TPR>
cudaError_t fwd_t(const LayerNormArgs& a, cudaStream_t s) {
    using C = Forward<T, VEC, NV, TPR>;
    static bool done[64] = {};
    if (!allow_smem(layer_norm_kernel<T, VEC, NV, TPR>, C::Fetch::SMEM, done)) return cudaErrorInvalidValue;
    const int grid = grid_rows(a.R, RowThreads<TPR>::ROWS, C::PER_SM);
    return launch_pdl(layer_norm_kernel<T, VEC, NV, TPR>, dim3(grid), dim3(C::THREADS), C::Fetch::SMEM, s, a.R, a.d,
                      static_cast<const T*>(a.x), a.x_stride, a.gamma, a.beta, a.eps, static_cast<T*>(a.y),
                      a.y_stride, a.mean_out, a.rstd_out);
}

template <typename T, int VEC>
cudaError_t fwd_v(const LayerNormArgs& a, cudaStream_t s) {
    const int d = a.d;
    // short rows: few columns a thread, or many would have none (us, against 16 columns of 8 or
    // 32 threads: 961280 BF16 rows of 16 at an odd pitch 158 -> 55, 143974 of 160 45 -> 27,
    // 51456 FP16 of 163 37 -> 22)
    if constexpr (VEC == 1) {
        if (d <= 8 * 4) return fwd_t<T, 1, 4, 8>(a, s);
        if (d <= 16 * 4) return fwd_t<T, 1, 4, 16>(a, s);
        if (d <= 16 * 8) return fwd_t<T, 1, 8, 16>(a, s);
        if (d <= 32 * 8) return fwd_t<T, 1, 8, 32>(a, s);
        if (d <= 32 * 12) return fwd_t<T, 1, 12, 32>(a, s);
    } else {
        if (d <= 8 * 8) return fwd_t<T, VEC, 8 / VEC, 8>(a, s);
        if (d <= 8 * 16) return fwd_t<T, VEC, 16 / VEC, 8>(a, s);
        if (d <= 16 * 16) return fwd_t<T, VEC, 16 / VEC, 16>(a, s);
    }
    if (d <= 32 * 16) return fwd_t<T, VEC, 16 / VEC, 32>(a, s);
    // a warp without a sync beats a CTA of four (32768 rows of 1024, BF16: 33 against 39 us)
    if constexpr (VEC > 1) {
        if (d <= 32 * 32) return fwd_t<T, VEC, 32 / VEC, 32>(a, s);
    } else {
        if (d <= 128 * 8) return fwd_t<T, 1, 8, 128>(a, s);
    }
    // CTAs of three quarters beside those of powers of two: fewer threads without columns,
    // and at 384 threads two CTAs an SM for one (BF16 rows of 2560, 5120, 100 MB: 61 -> 49,
    // 68 -> 51 us)
    if (d <= 96 * 16) return fwd_t<T, VEC, 16 / VEC, 96>(a, s);
    if (d <= 128 * 16) return fwd_t<T, VEC, 16 / VEC, 128>(a, s);
    if (d <= 192 * 16) return fwd_t<T, VEC, 16 / VEC, 192>(a, s);
    if (d <= 256 * 16) return fwd_t<T, VEC, 16 / VEC, 256>(a, s);
    if (d <= 384 * 16) return fwd_t<T, VEC, 16 / VEC, 384>(a, s);
    if (d <= 512 * 16) return fwd_t<T, VEC, 16 / VEC, 512>(a, s);
    return fwd_t<T, VEC, 16 / VEC, 1024>(a, s);
}

template <typename T>
cudaError_t fwd_d(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (a.d > FWD_MAX_D)
        return launch_pdl(layer_norm_long_kernel<T>, dim3(grid_rows(a.R, 1, 2)), dim3(1024), 0, s, a.R, a.d,
                          static_cast<const T*>(a.x), a.x_stride, a.gamma, a.beta, a.eps, static_cast<T*>(a.y),
                          a.y_stride, a.mean_out, a.rstd_out);
    if (a.d % V == 0 && vec_ok(a.x, a.x_stride, sizeof(T)) && vec_ok(a.y, a.y_stride, sizeof(T)) &&
        vec_ok(a.gamma, 0, 4) && vec_ok(a.beta, 0, 4))
        return fwd_v<T, V>(a, s);
    return fwd_v<T, 1>(a, s);
}

template <typename T, int VEC, int NV, int TPR>
cudaError_t bwd_t(const LayerNormArgs& a, int grid, float* part, cudaStream_t s) {
    using C = Backward<T, VEC, NV, TPR>;
    constexpr int SMEM = 2 * C::Fetch::SMEM;
    static bool done[64] = {};
    if (!allow_smem(layer_norm_bwd_kernel<T, VEC, NV, TPR>, SMEM, done)) return cudaErrorInvalidValue;
    return launch_pdl(layer_norm_bwd_kernel<T, VEC, NV, TPR>, dim3(grid), dim3(C::THREADS), SMEM, s, a.R, a.d,
                      static_cast<const T*>(a.dy), a.dy_stride, static_cast<const T*>(a.x), a.x_stride, a.mean,
                      a.rstd, a.gamma, static_cast<T*>(a.y), a.y_stride, part);
}

template <typename T, int VEC>
cudaError_t bwd_v(const LayerNormArgs& a, int grid, float* part, cudaStream_t s) {
    switch (bwd_threads(a.d)) {
        case 8:
            if constexpr (VEC == 1)
                if (a.d <= 8 * 4) return bwd_t<T, 1, 4, 8>(a, grid, part, s);
            return bwd_t<T, VEC, 8 / VEC, 8>(a, grid, part, s);
        case 16: return bwd_t<T, VEC, 8 / VEC, 16>(a, grid, part, s);
        case 32:
            if (a.d <= 32 * 8) return bwd_t<T, VEC, 8 / VEC, 32>(a, grid, part, s);
            // elements one by one: as few columns a thread as there are
            if constexpr (VEC == 1)
                if (a.d <= 32 * 12) return bwd_t<T, 1, 12, 32>(a, grid, part, s);
            return bwd_t<T, VEC, 16 / VEC, 32>(a, grid, part, s);
        case 128:
            if (a.d <= 128 * 8) return bwd_t<T, VEC, 8 / VEC, 128>(a, grid, part, s);
            if constexpr (VEC == 1)  // 17835 FP32 rows of 1411 80 -> 72 us
                if (a.d <= 128 * 12) return bwd_t<T, 1, 12, 128>(a, grid, part, s);
            return bwd_t<T, VEC, 16 / VEC, 128>(a, grid, part, s);
        case 192: return bwd_t<T, VEC, 16 / VEC, 192>(a, grid, part, s);
        case 256: return bwd_t<T, VEC, 16 / VEC, 256>(a, grid, part, s);
        case 384: return bwd_t<T, VEC, 16 / VEC, 384>(a, grid, part, s);
        default: return bwd_t<T, VEC, 16 / VEC, 512>(a, grid, part, s);
    }
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
               vec_ok(a.y, a.y_stride, sizeof(T)) && vec_ok(a.gamma, 0, 4)) {
        e = bwd_v<T, V>(a, n, part, s);
    } else {
        e = bwd_v<T, 1>(a, n, part, s);
    }
    if (e != cudaSuccess || part == nullptr) return e;
    return launch_pdl(layer_norm_cols_sum_kernel, dim3((2 * a.d + 31) / 32), dim3(32 * COL_ROWS), 0, s, n, a.d,
                      static_cast<const float*>(part), a.dgamma, a.dbeta);
}

}  // namespace

int layer_norm_bwd_parts(int R, int d) {
    if (d > BWD_MAX_D) return R < 16 ? R : 16;
    const int t = bwd_threads(d);
    return grid_rows(R, t <= 32 ? 128 / t : 1, bwd_per_sm(t));
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
