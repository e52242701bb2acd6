// Element types of the operators around the layer (FP32, BF16, FP16): vector
// loads to FP32, vector stores rounded once to nearest-even, and the warp and
// CTA sums they share.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

template <typename T>
MOE_DEV float to_f32(T v);
template <>
MOE_DEV float to_f32<float>(float v) { return v; }
template <>
MOE_DEV float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
MOE_DEV float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T>
MOE_DEV T from_f32(float v);
template <>
MOE_DEV float from_f32<float>(float v) { return v; }
template <>
MOE_DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
MOE_DEV __half from_f32<__half>(float v) { return __float2half_rn(v); }

// VEC consecutive elements as loaded: one 16-byte word, or one element.
template <typename T, int VEC>
struct Raw {
    static_assert(VEC * sizeof(T) == 16, "a vector is 16 bytes");
    uint4 v;
    MOE_DEV void load(const T* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    MOE_DEV void clear() { v = make_uint4(0, 0, 0, 0); }
    MOE_DEV void get(float (&f)[VEC]) const {
        const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = to_f32(e[i]);
    }
    MOE_DEV void set(const float (&f)[VEC]) {
        T* e = reinterpret_cast<T*>(&v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = from_f32<T>(f[i]);
    }
    MOE_DEV void store(T* p) const { *reinterpret_cast<uint4*>(p) = v; }
};
template <typename T>
struct Raw<T, 1> {
    T v;
    MOE_DEV void load(const T* p) { v = *p; }
    MOE_DEV void clear() { v = from_f32<T>(0.0f); }
    MOE_DEV void get(float (&f)[1]) const { f[0] = to_f32(v); }
    MOE_DEV void set(const float (&f)[1]) { v = from_f32<T>(f[0]); }
    MOE_DEV void store(T* p) const { *p = v; }
};

// sigmoid(v) = exp(v) / (1 + exp(v)) below zero, where exp(-v) would leave
// FP32's range while v sigmoid(v) is still in it. On the special-function
// unit: the argument |v| log2(e) keeps what its rounding lost (and what log2(e)
// itself does), so that the result is off by 4 units of 2^-23 down to v = -87, and
// below that, where it is subnormal, by a unit of 2^-149 besides.
MOE_DEV float sigmoid_f(float v) {
    constexpr double LOG2E = 1.4426950408889634;
    constexpr float HI = static_cast<float>(LOG2E), LO = static_cast<float>(LOG2E - static_cast<double>(HI));
    const float a = fminf(fabsf(v), 150.0f), t = a * -HI;  // below 2^-150 is zero
    const float lost = fmaf(a, -LO, fmaf(a, -HI, -t));
    float e, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    e = fmaf(e, lost * 0.6931471805599453f, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return (v >= 0.0f ? 1.0f : e) * r;
}

// SiLU's sigmoid in the output's precision: 16-bit outputs take the fast
// exponential and division, off by (4 + 1.2 |v|) units of 2^-23 at most down to
// v = -87 (8-bit gate/up product of 131072 rows 1012 us with the other one, 992 with this).
template <typename O>
MOE_DEV float sigmoid_to(float v) {
    if constexpr (sizeof(O) == 4) return sigmoid_f(v);
    const float e = __expf(-fabsf(v));
    return __fdividef(v >= 0.0f ? 1.0f : e, 1.0f + e);
}

// Sum over the TPR <= 32 threads of a row, the same in all of them.
template <int TPR>
MOE_DEV float seg_sum(float v) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum of the W <= 32 values that lanes 0 to W - 1 hold (the lanes behind: 0), the
// same in every lane and in a fixed order.
template <int W>
MOE_DEV float group_sum(float v) {
    constexpr int P = W > 16 ? 32 : W > 8 ? 16 : W > 4 ? 8 : W > 2 ? 4 : W;
#pragma unroll
    for (int o = P / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (W < 32) v = __shfl_sync(0xffffffffu, v, 0);
    return v;
}

// Sums of a and b over the TPR threads of a row, the same in all of them and
// in a fixed order. TPR <= 32: within the warp. Else over the CTA (TPR
// threads), through `scratch`, two halves of 2 * TPR / 32 floats used in turn:
// the sync of one call orders the reads of the call before last.
template <int TPR>
MOE_DEV void row_sum2(float& a, float& b, float* scratch, int& turn) {
    a = seg_sum<(TPR < 32 ? TPR : 32)>(a);
    b = seg_sum<(TPR < 32 ? TPR : 32)>(b);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        float* s = scratch + (turn & 1) * 2 * W;
        ++turn;
        const int w = threadIdx.x >> 5;
        if (lane_id() == 0) {
            s[w] = a;
            s[W + w] = b;
        }
        __syncthreads();
        const int l = static_cast<int>(lane_id());
        a = group_sum<W>(l < W ? s[l] : 0.0f);
        b = group_sum<W>(l < W ? s[W + l] : 0.0f);
    }
}

// The same of one value; scratch: two halves of TPR / 32 floats.
template <int TPR>
MOE_DEV void row_sum(float& a, float* scratch, int& turn) {
    a = seg_sum<(TPR < 32 ? TPR : 32)>(a);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        float* s = scratch + (turn & 1) * W;
        ++turn;
        if (lane_id() == 0) s[threadIdx.x >> 5] = a;
        __syncthreads();
        const int l = static_cast<int>(lane_id());
        a = group_sum<W>(l < W ? s[l] : 0.0f);
    }
}

// Two FP32 values in a register pair; the packed operations do both at the
// issue of one.
struct F2 {
    unsigned long long v;
};
MOE_DEV F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
MOE_DEV void unpack(F2 p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v)); }
MOE_DEV float both(F2 p) {
    float a, b;
    unpack(p, a, b);
    return a + b;
}
MOE_DEV F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
MOE_DEV F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
MOE_DEV F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

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

// The k-th pair of a thread's columns less m, zeros (as loaded) past the row's end. Of a row of large values
// without any variance (v - m) r would pass FP32's range there, and take the row's sums with it.
template <int VEC, int TPR>
MOE_DEV F2 less(F2 v, float m, int k, int d, int t) {
    const float a = (2 * k / VEC * TPR + t) * VEC < d ? -m : 0.0f;
    return add2(v, f2(a, VEC > 1 ? a : ((2 * k + 1) * TPR + t < d ? -m : 0.0f)));
}

// VEC consecutive floats (16-byte aligned where VEC >= 4).
template <int VEC>
MOE_DEV void load_f32(const float* p, float (&f)[VEC]) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
            f[i] = v.x;
            f[i + 1] = v.y;
            f[i + 2] = v.z;
            f[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = __ldg(p + i);
    }
}

template <int VEC>
MOE_DEV void store_f32(float* p, const float (&f)[VEC]) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = f[i];
    }
}

MOE_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MOE_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// What a thread reads of the rows ahead: its own vectors (NV per row, vector i
// at column (i * TPR + t) * VEC), copied asynchronously into its own part of
// shared memory, D rows deep, so that the bytes in flight do not depend on
// registers and no thread waits for another's copies. Elements that cp.async
// cannot move (single 16-bit ones) go through registers, one row ahead.
template <typename T, int VEC, int NV, int TPR, int THREADS, int DEPTH>
struct RowFetch {
    static constexpr int BYTES = VEC * static_cast<int>(sizeof(T));
    static constexpr bool ASYNC = BYTES >= 4;
    static constexpr int D = ASYNC ? DEPTH : 1;
    static constexpr int SMEM = ASYNC ? D * NV * THREADS * BYTES : 0;
    T* slots;
    const T* base;
    long long pitch;
    int d, t;
    Raw<T, VEC> ahead[ASYNC ? 1 : NV];

    MOE_DEV void init(void* smem, const T* base_, long long pitch_, int d_, int t_) {
        slots = static_cast<T*>(smem) + threadIdx.x * VEC;
        base = base_;
        pitch = pitch_;
        d = d_;
        t = t_;
    }
    // Starts the copies of `row` into slot s (nothing unless there).
    MOE_DEV void issue(int s, long long row, bool there) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (there && c < d) {
                if constexpr (ASYNC) {
                    T* at = slots + (s * NV + i) * THREADS * VEC;
                    if constexpr (BYTES == 16) cp_async_16(at, base + row * pitch + c);
                    else cp_async_4(at, base + row * pitch + c);
                } else {
                    ahead[i].load(base + row * pitch + c);
                }
            }
        }
    }
    // Slot s as FP32 pairs, vectors one after the other (zeros past the row's end).
    MOE_DEV void pairs(int s, F2 (&p)[NV * VEC / 2]) const {
        float f[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) get(s, i, f[i]);
#pragma unroll
        for (int k = 0; k < NV * VEC / 2; ++k) p[k] = f2(f[2 * k / VEC][2 * k % VEC], f[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
    }
    // Vector i of slot s as loaded, or as FP32 (zeros past the row's end).
    MOE_DEV Raw<T, VEC> raw(int s, int i) const {
        const bool in = (i * TPR + t) * VEC < d;
        Raw<T, VEC> r;
        r.clear();
        if constexpr (ASYNC) {
            if (in) r = *reinterpret_cast<const Raw<T, VEC>*>(slots + (s * NV + i) * THREADS * VEC);
        } else {
            if (in) r = ahead[i];
        }
        return r;
    }
    MOE_DEV void get(int s, int i, float (&f)[VEC]) const { raw(s, i).get(f); }
};

// How the row kernels lay rows over threads: TPR threads a row, up to a warp
// several rows to a CTA of 128.
template <int TPR>
struct RowThreads {
    static constexpr int THREADS = TPR <= 32 ? 128 : TPR;
    static constexpr int ROWS = THREADS / TPR;      // rows a CTA works on at a time
    MOE_DEV static int col() { return static_cast<int>(threadIdx.x) % TPR; }
    MOE_DEV static int row() { return static_cast<int>(threadIdx.x) / TPR; }
    // the first of the rows that the warp (or the CTA) works on together, from this thread's
    MOE_DEV static long long first(long long row) { return TPR < 32 ? row - static_cast<int>(lane_id()) / TPR : row; }
};

// CTAs for `rows` rows, rpc of them at a time, at most per_sm on an SM.
inline int grid_rows(long long rows, int rpc, int per_sm) {
    const long long want = (rows + rpc - 1) / rpc, cap = static_cast<long long>(num_sms()) * per_sm;
    return static_cast<int>(want < cap ? want : cap);
}

// Dynamic shared memory above the default limit has to be asked for, once per
// kernel and device.
template <typename K>
inline bool allow_smem(K kernel, int bytes, bool (&done)[64]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (!done[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
        done[dev] = true;
    }
    return true;
}

}  // namespace moe
