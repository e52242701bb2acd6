// Low-rank adapters (adapter.cu has the formula): what the kernels of few rows and of many
// share. Tiles of a group's positions, the inner values' pieces, rows of base and out.
#pragma once

#include <algorithm>

#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int MAXE = 1024;
constexpr int THREADS = 256;

// Tiles of TM positions: how many come before each group, and where a group begins.
// Group E is what has no adapter.
struct Groups {
    int tp[MAXE + 2], lo[MAXE + 2];
};

// Fills the table (all threads of the CTA; ends with a sync) and returns the number of
// tiles. Offsets are clamped to [0, T]; a group that ends before it begins is empty.
template <int TM>
MOE_DEV int group_table(const AdapterArgs& a, bool rest, Groups& g) {
    __shared__ int wsum[THREADS / 32];
    constexpr int PER = (MAXE + 1 + THREADS - 1) / THREADS;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int G = a.E + 1, per = (G + THREADS - 1) / THREADS;
    int lo[PER], c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = t * per + i;
        lo[i] = c[i] = 0;
        if (i < per && e < G) {
            lo[i] = min(max(__ldg(a.offsets + e), 0), a.T);
            const int hi = e < a.E ? min(max(__ldg(a.offsets + e + 1), 0), a.T) : (rest ? a.T : lo[i]);
            c[i] = hi > lo[i] ? (hi - lo[i] + TM - 1) / TM : 0;
            g.lo[e] = lo[i];
        }
        sum += c[i];
    }
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) wsum[w] = x;
    __syncthreads();
    int before = x - sum, total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        before += i < w ? wsum[i] : 0;
        total += wsum[i];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = t * per + i;
        if (i < per && e < G) g.tp[e] = before;
        before += c[i];
    }
    if (t == 0) {
        g.tp[G] = total;
        g.lo[G] = a.T;
    }
    __syncthreads();
    return total;
}

// CTAs with so many bytes of dynamic shared memory that an SM holds (the registers leave two): of its 228 KB
// each takes 1 KB more, and the table above with less than 512 bytes of other variables.
constexpr int ctas_an_sm(size_t smem) { return smem + sizeof(Groups) + 512 + 1024 <= (228 << 10) / 2 ? 2 : 1; }

struct Tile {
    int e, pos, n;  // group, first position, positions
};
template <int TM>
MOE_DEV Tile tile_of(int u, const AdapterArgs& a, const Groups& g) {
    int lo = 0, hi = a.E + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.tp[mid] <= u) lo = mid;
        else hi = mid;
    }
    Tile t;
    t.e = lo;
    t.pos = g.lo[lo] + (u - g.tp[lo]) * TM;
    t.n = min(TM, g.lo[lo + 1] - t.pos);  // a group ends where the next begins
    return t;
}

// The row that position i stands for, -1 where the index names none.
MOE_DEV int row_of(const AdapterArgs& a, int i) {
    const int r = a.rows != nullptr ? __ldg(a.rows + i) : i;
    return r >= 0 && r < a.T ? r : -1;
}

// v in pieces of T that add up to it: 3 for FP32 outputs (its 24 bits), 2 for 16-bit ones. BF16's two
// leave at most 2^-16 of v out, a 256th of what rounding base, and then the output, to BF16 may (the third:
// 8192 rows of 4, 4096 x 4096, rank 64, 60 -> 70 us, 16384 of rank 16 60 -> 62); FP16's 2^-22. FP16 first takes
// a row to below 2^15 by a power of two.
template <typename T>
MOE_DEV uint32_t pack2(T x, T y) {
    return static_cast<uint32_t>(*reinterpret_cast<unsigned short*>(&x)) |
           static_cast<uint32_t>(*reinterpret_cast<unsigned short*>(&y)) << 16;
}
template <typename T, int NP>
MOE_DEV void split(float v, T (&p)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        p[i] = from_f32<T>(v);
        const float f = to_f32(p[i]);
        v = fabsf(f) <= 3.4e38f ? v - f : 0.0f;  // nothing is left of an infinity or a NaN
    }
}

// Pieces of v against an infinite element of B: their products have different signs, or one is 0 inf,
// and the sum is NaN where v B^T is an infinity. So 8 consecutive columns of a row whose sums hold a NaN
// are not stored but taken again, from v whole: v(k) of the row, rows of B r apart. A NaN in v stays
// what it is (the first one ends the loop). Behind all stores of a block, so that these wait for no
// branch (at each store: 16384 x 2048 x 2816, rank 16, 82 us for 58).
MOE_DEV bool any_nan(const F2 (&acc)[4]) {
    const float s = both(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])));
    return s != s;
}
template <typename T, typename V>
MOE_DEV void sums_again(float (&s)[8], V v, const T* b, int r, int columns) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.0f;
#pragma unroll 1
    for (int k = 0; k < r; ++k) {
        const float x = v(k);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < columns) s[j] = fmaf(x, to_f32(b[static_cast<long long>(j) * r + k]), s[j]);
        if (x != x) return;
    }
}
template <typename T, typename O, typename V>
MOE_DEV void store_again(O* to, const O* base, V v, const T* b, int r, float back) {
    float s[8];
    sums_again(s, v, b, r, 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) to[j] = from_f32<O>(fmaf(s[j], back, base != nullptr ? to_f32(base[j]) : 0.0f));
}

// 8 consecutive elements of base as loaded (16-byte aligned, all or none).
template <typename O>
struct Cols {
    static constexpr int N = 8 * sizeof(O) / 16, W = 8 / N;
    Raw<O, W> v[N];
    MOE_DEV void load(const O* p, bool there) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i].clear();
            if (there) v[i].v = *reinterpret_cast<const uint4*>(p + i * W);  // base may be out: no read-only loads
        }
    }
    // acc times `by`, added to these elements and stored, two at a time.
    MOE_DEV void add_to(O* p, const F2 (&acc)[4], float by) const {
        const F2 s = f2(by, by);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float e[W];
            v[i].get(e);
#pragma unroll
            for (int q = 0; q < W; q += 2) unpack(fma2(acc[(i * W + q) / 2], s, f2(e[q], e[q + 1])), e[q], e[q + 1]);
            Raw<O, W> o;
            o.set(e);
            o.store(p + i * W);
        }
    }
    MOE_DEV void copy_to(O* p) const {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i].store(p + i * W);
    }
};

// Asynchronous copies of 16 or 8 bytes, zeros where there is nothing to copy.
MOE_DEV void cp_async_16z(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
MOE_DEV void cp_async_8z(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(there ? 8 : 0) : "memory");
}

// The sum of the slices of 4 consecutive inner values.
MOE_DEV float4 inner4(const AdapterArgs& a, int pos, int k, int slices) {
    const float* v = a.v + static_cast<long long>(pos) * a.rp + k;
    const long long plane = static_cast<long long>(a.T) * a.rp;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < slices; i += 8) {
        float4 o[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            o[q] = i + q < slices ? *reinterpret_cast<const float4*>(v + (i + q) * plane) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            s.x += o[q].x;
            s.y += o[q].y;
            s.z += o[q].z;
            s.w += o[q].w;
        }
    }
    return s;
}
MOE_DEV float largest_finite(float4 v, float most) {
    for (float f : {v.x, v.y, v.z, v.w})
        if (fabsf(f) <= 3.4e38f) most = fmaxf(most, fabsf(f));
    return most;
}
// 2^(14 - e) for a largest value of [2^e, 2^(e + 1)), and its inverse.
MOE_DEV void row_scale(float most, float& scale, float& back) {
    const int e = min(max(14 + 127 - static_cast<int>(__float_as_uint(most) >> 23), -126), 126);
    scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    back = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

MOE_DEV float4 ld_shared_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

}  // namespace
}  // namespace moe
