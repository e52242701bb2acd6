// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + s_e (x[t] A_e^T) B_e^T,   e the adapter of row t
//
// Rows come grouped by adapter: group e is the positions offsets[e] to offsets[e + 1]
// of `rows`; positions from offsets[E] on have no adapter. Two launches: the first
// computes v = s_e x[t] A_e^T into the workspace (by position, FP32), the second adds
// v B_e^T to base.
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
    // a group's end is the next one's begin (offsets ascend); the last tile of one may be short
    const int end = lo < a.E ? min(max(__ldg(a.offsets + lo + 1), 0), a.T) : a.T;
    Tile t;
    t.e = lo;
    t.pos = g.lo[lo] + (u - g.tp[lo]) * TM;
    t.n = min(TM, end - t.pos);
    return t;
}

// The row that position i stands for, -1 where the index names none.
MOE_DEV int row_of(const AdapterArgs& a, int i) {
    const int r = a.rows != nullptr ? __ldg(a.rows + i) : i;
    return r >= 0 && r < a.T ? r : -1;
}

// ---------------------------------------------------------------------------
// any type, width, rank and alignment
// ---------------------------------------------------------------------------
constexpr int SH_ROWS = 4, SH_RANKS = 8;        // of a warp
constexpr int SH_TILE = SH_ROWS * THREADS / 32;

template <typename T>
__global__ void __launch_bounds__(THREADS) adapter_shrink_kernel(const __grid_constant__ AdapterArgs a) {
    __shared__ Groups g;
    pdl_wait();
    pdl_trigger();
    const int tiles = group_table<SH_TILE>(a, false, g);
    const int lane = static_cast<int>(lane_id()), w = threadIdx.x >> 5;
    const int rb = (a.r + SH_RANKS - 1) / SH_RANKS;
    const T* x = static_cast<const T*>(a.x);
    for (long long u = blockIdx.x; u < static_cast<long long>(tiles) * rb; u += gridDim.x) {
        const Tile t = tile_of<SH_TILE>(static_cast<int>(u / rb), a, g);
        const int j0 = static_cast<int>(u % rb) * SH_RANKS;
        const int p0 = t.pos + w * SH_ROWS;
        if (p0 >= t.pos + t.n) continue;
        const T* A = static_cast<const T*>(a.a) + (static_cast<long long>(t.e) * a.r + j0) * a.d;
        const T* xr[SH_ROWS];
#pragma unroll
        for (int i = 0; i < SH_ROWS; ++i) {
            const int r = p0 + i < t.pos + t.n ? row_of(a, p0 + i) : 0;
            if (r < 0 && lane == 0) atomicOr(a.err, ERRBIT_INDEX);
            xr[i] = x + max(r, 0) * a.x_stride;
        }
        float acc[SH_ROWS][SH_RANKS] = {};
        for (int k = lane; k < a.d; k += 32) {
            float xv[SH_ROWS];
#pragma unroll
            for (int i = 0; i < SH_ROWS; ++i) xv[i] = to_f32(xr[i][k]);
#pragma unroll
            for (int j = 0; j < SH_RANKS; ++j) {
                const float av = j0 + j < a.r ? to_f32(A[static_cast<long long>(j) * a.d + k]) : 0.0f;
#pragma unroll
                for (int i = 0; i < SH_ROWS; ++i) acc[i][j] = fmaf(xv[i], av, acc[i][j]);
            }
        }
        const float s = a.scale != nullptr ? __ldg(a.scale + t.e) : 1.0f;
#pragma unroll
        for (int i = 0; i < SH_ROWS; ++i)
#pragma unroll
            for (int j = 0; j < SH_RANKS; ++j) {
                const float v = seg_sum<32>(acc[i][j]);
                if (lane == 0 && p0 + i < t.pos + t.n && j0 + j < a.r)
                    a.v[static_cast<long long>(p0 + i) * a.r + j0 + j] = s * v;
            }
    }
}

constexpr int EX_TILE = 16, EX_RANKS = 16;

template <typename T, typename O>
__global__ void __launch_bounds__(THREADS) adapter_expand_kernel(const __grid_constant__ AdapterArgs a) {
    __shared__ Groups g;
    __shared__ __align__(16) float sv[EX_TILE][EX_RANKS];
    __shared__ int srow[EX_TILE];
    pdl_wait();
    pdl_trigger();
    const int tiles = group_table<EX_TILE>(a, !a.in_place, g);
    const int nb = (a.N + THREADS - 1) / THREADS;
    const O* base = static_cast<const O*>(a.base);
    O* out = static_cast<O*>(a.out);
    for (long long u = blockIdx.x; u < static_cast<long long>(tiles) * nb; u += gridDim.x) {
        const Tile t = tile_of<EX_TILE>(static_cast<int>(u / nb), a, g);
        const int n = static_cast<int>(u % nb) * THREADS + threadIdx.x;
        __syncthreads();
        if (threadIdx.x < EX_TILE) srow[threadIdx.x] = threadIdx.x < t.n ? row_of(a, t.pos + threadIdx.x) : -1;
        float acc[EX_TILE] = {};
        for (int j0 = 0; t.e < a.E && j0 < a.r; j0 += EX_RANKS) {
            __syncthreads();
            for (int i = threadIdx.x; i < EX_TILE * EX_RANKS; i += THREADS) {
                const int row = i / EX_RANKS, j = j0 + i % EX_RANKS;
                sv[row][i % EX_RANKS] = row < t.n && j < a.r ? a.v[static_cast<long long>(t.pos + row) * a.r + j] : 0.0f;
            }
            float b[EX_RANKS];
            const T* B = static_cast<const T*>(a.b) + (static_cast<long long>(t.e) * a.N + n) * a.r + j0;
#pragma unroll
            for (int j = 0; j < EX_RANKS; ++j) b[j] = n < a.N && j0 + j < a.r ? to_f32(B[j]) : 0.0f;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < EX_TILE; ++i)
#pragma unroll
                for (int j = 0; j < EX_RANKS; ++j)
                    if (j0 + j < a.r) acc[i] = fmaf(sv[i][j], b[j], acc[i]);
        }
        __syncthreads();
        if (n >= a.N) continue;
        for (int i = 0; i < t.n; ++i) {
            const int row = srow[i];
            if (row < 0) continue;
            float v = base != nullptr ? to_f32(base[row * a.base_stride + n]) : 0.0f;
            if (t.e < a.E) v += acc[i];
            out[row * a.out_stride + n] = from_f32<O>(v);
        }
    }
}

// ---------------------------------------------------------------------------
// 16-bit types: matrix instructions on fragments that come straight from memory
// ---------------------------------------------------------------------------
// m16n8k16: lane (g, t) = (lane / 4, lane % 4) holds rows g and g + 8 of A, column g of B, at
// four of the 16 reduction indices, the same four for A and B; which four is free. Taken as
// consecutive ones, a lane's fragments of one or two instructions are one load.
template <typename T>
MOE_DEV void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (sizeof(T) == 2 && __is_same(T, __half))
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// n <= 8 (4) elements from p, the rest zeros: one load where they are aligned.
template <typename T, bool VEC>
MOE_DEV uint4 load8(const T* p, int n) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if constexpr (VEC) {
        if (n > 0) v = __ldg(reinterpret_cast<const uint4*>(p));
    } else {
        uint32_t w[4] = {0, 0, 0, 0};
        const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i / 2] |= static_cast<uint32_t>(__ldg(q + i)) << (16 * (i & 1));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}
template <typename T, bool VEC>
MOE_DEV uint2 load4(const T* p, int n) {
    uint2 v = make_uint2(0, 0);
    if constexpr (VEC) {
        if (n > 0) v = __ldg(reinterpret_cast<const uint2*>(p));
    } else {
        uint32_t w[2] = {0, 0};
        const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) w[i / 2] |= static_cast<uint32_t>(__ldg(q + i)) << (16 * (i & 1));
        v = make_uint2(w[0], w[1]);
    }
    return v;
}

// v = s x A^T of 16 MT positions by 8 NT ranks and one slice of d: the CTA's warps take
// every eighth 32 of the slice, and their sums are added in order.
//   a.v [slices][T][rp], rp = r rounded up to 16 and the ranks behind r zero.
template <int MT, int NT>
struct Shrink {
    // chunks of 32 a warp has in flight, as registers allow
    static constexpr int AHEAD = 2 * MT + NT <= 4 ? 4 : 2 * MT + NT <= 10 ? 2 : 1;
};
template <typename T, int MT, int NT, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) adapter_shrink_mma_kernel(const __grid_constant__ AdapterArgs a) {
    constexpr int WARPS = THREADS / 32, U = Shrink<MT, NT>::AHEAD;
    __shared__ Groups g;
    __shared__ float red[WARPS][NT * 4][32];
    pdl_wait();
    pdl_trigger();
    const int tiles = group_table<16 * MT>(a, false, g);
    const int lane = static_cast<int>(lane_id()), w = threadIdx.x >> 5, gi = lane >> 2, ti = lane & 3;
    const int rb = (a.rp + 8 * NT - 1) / (8 * NT), parts = rb * a.slices;
    const int len = ((a.d + a.slices - 1) / a.slices + 31) / 32 * 32;
    const T* x = static_cast<const T*>(a.x);
    for (long long u = blockIdx.x; u < static_cast<long long>(tiles) * parts; u += gridDim.x) {
        const Tile t = tile_of<16 * MT>(static_cast<int>(u / parts), a, g);
        const int part = static_cast<int>(u % parts), j0 = part % rb * 8 * NT, slice = part / rb;
        const int k0 = slice * len, k1 = min(a.d, k0 + len);
        const T* xr[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 16 * m + 8 * h + gi;
                xr[m][h] = nullptr;
                if (i < t.n) {
                    const int r = row_of(a, t.pos + i);
                    if (r >= 0) xr[m][h] = x + r * a.x_stride;
                    else if (ti == 0) atomicOr(a.err, ERRBIT_INDEX);
                }
            }
        const T* A = static_cast<const T*>(a.a) + static_cast<long long>(t.e) * a.r * a.d;
        float acc[MT][NT][4] = {};
        for (int k = k0 + 32 * w; k < k1; k += 32 * WARPS * U) {
            uint4 fx[U][MT][2], fa[U][NT];
#pragma unroll
            for (int c = 0; c < U; ++c) {
                const int at = k + 32 * WARPS * c + 8 * ti, n = k1 - at;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) fx[c][m][h] = load8<T, VEC>(xr[m][h] + at, xr[m][h] != nullptr ? n : 0);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int rank = j0 + 8 * j + gi;
                    fa[c][j] = load8<T, VEC>(A + static_cast<long long>(rank) * a.d + at, rank < a.r ? n : 0);
                }
            }
#pragma unroll
            for (int c = 0; c < U; ++c)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        mma16816<T>(acc[m][j], fx[c][m][0].x, fx[c][m][1].x, fx[c][m][0].y, fx[c][m][1].y, fa[c][j].x, fa[c][j].y);
                        mma16816<T>(acc[m][j], fx[c][m][0].z, fx[c][m][1].z, fx[c][m][0].w, fx[c][m][1].w, fa[c][j].z, fa[c][j].w);
                    }
        }
        const float s = a.scale != nullptr ? __ldg(a.scale + t.e) : 1.0f;
        float* out = a.v + static_cast<long long>(slice) * a.T * a.rp;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) red[w][4 * j + i][lane] = acc[m][j][i];
            __syncthreads();
            for (int i = threadIdx.x; i < NT * 128; i += THREADS) {
                const int q = i >> 5, l = i & 31;
                float v = red[0][q][l];
#pragma unroll
                for (int o = 1; o < WARPS; ++o) v += red[o][q][l];
                const int p = 16 * m + 8 * (q >> 1 & 1) + (l >> 2), rank = j0 + 8 * (q >> 2) + 2 * (l & 3) + (q & 1);
                if (p < t.n && rank < a.rp) out[static_cast<long long>(t.pos + p) * a.rp + rank] = rank < a.r ? s * v : 0.0f;
            }
            __syncthreads();
        }
    }
}

// v in pieces of T that add up to it: 2 for 16-bit outputs (bf16: 16 bits of v), 3 for FP32.
// FP16 first takes a row to below 2^15 by a power of two.
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

// out = base + v B^T of 16 MT positions by a range of columns. A warp takes 32 columns at a
// time: column 2 i + c of its instruction j stands for column 8 i + 2 j + c, so that a lane
// ends with 8 consecutive columns of its two rows.
template <typename T, typename O, int MT, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) adapter_expand_mma_kernel(const __grid_constant__ AdapterArgs a) {
    constexpr int WARPS = THREADS / 32, NP = sizeof(O) == 4 ? 3 : 2, ROWS = 16 * MT;
    constexpr bool SCALED = __is_same(T, __half);
    __shared__ Groups g;
    __shared__ int srow[ROWS];
    __shared__ float sscale[SCALED ? ROWS : 1];
    extern __shared__ __align__(16) uint4 frag[];  // [rp / 16][NP][MT][32]
    pdl_wait();
    pdl_trigger();
    const int tiles = group_table<ROWS>(a, !a.in_place, g);
    const int lane = static_cast<int>(lane_id()), w = threadIdx.x >> 5, gi = lane >> 2, ti = lane & 3;
    const int KS = a.rp / 16, nb = a.col_parts, len = ((a.N + nb - 1) / nb + 31) / 32 * 32;
    const O* base = static_cast<const O*>(a.base);
    O* out = static_cast<O*>(a.out);
    const long long plane = static_cast<long long>(a.T) * a.rp;
    auto inner = [&](int p, int k) {
        const float* v = a.v + static_cast<long long>(p) * a.rp + k;
        float4 s = *reinterpret_cast<const float4*>(v);
        for (int i = 1; i < a.slices; ++i) {
            const float4 o = *reinterpret_cast<const float4*>(v + i * plane);
            s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w;
        }
        return s;
    };
    for (long long u = blockIdx.x; u < static_cast<long long>(tiles) * nb; u += gridDim.x) {
        const Tile t = tile_of<ROWS>(static_cast<int>(u / nb), a, g);
        const int c0 = static_cast<int>(u % nb) * len, c1 = min(a.N, c0 + len);
        const bool adapted = t.e < a.E;
        __syncthreads();
        if (threadIdx.x < ROWS) srow[threadIdx.x] = threadIdx.x < t.n ? row_of(a, t.pos + threadIdx.x) : -1;
        if (adapted) {
            if constexpr (SCALED) {
                constexpr int PER = THREADS / ROWS;  // threads a row, within a warp
                const int row = threadIdx.x / PER;
                float m = 0.0f;
                for (int k = threadIdx.x % PER * 4; row < t.n && k < a.rp; k += PER * 4) {
                    const float4 v = inner(t.pos + row, k);
                    for (float f : {v.x, v.y, v.z, v.w})
                        if (fabsf(f) <= 3.4e38f) m = fmaxf(m, fabsf(f));
                }
#pragma unroll
                for (int o = PER / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                // 2^(14 - e) for a largest value of [2^e, 2^(e + 1))
                const int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
                if (threadIdx.x % PER == 0) sscale[row] = __uint_as_float(static_cast<uint32_t>(min(max(14 - e, -126), 126) + 127) << 23);
                __syncthreads();
            }
            for (int i = threadIdx.x; i < KS * MT * 32; i += THREADS) {
                const int l = i & 31, m = i / 32 % MT, ks = i / (32 * MT), k = 16 * ks + 4 * (l & 3);
                T q[2][4][NP];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = 16 * m + 8 * h + (l >> 2);
                    float4 v = p < t.n ? inner(t.pos + p, k) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if constexpr (SCALED) {
                        const float f = sscale[p];
                        v.x *= f; v.y *= f; v.z *= f; v.w *= f;
                    }
                    split<T, NP>(v.x, q[h][0]);
                    split<T, NP>(v.y, q[h][1]);
                    split<T, NP>(v.z, q[h][2]);
                    split<T, NP>(v.w, q[h][3]);
                }
#pragma unroll
                for (int o = 0; o < NP; ++o)
                    frag[((ks * NP + o) * MT + m) * 32 + l] =
                        make_uint4(pack2(q[0][0][o], q[0][1][o]), pack2(q[1][0][o], q[1][1][o]), pack2(q[0][2][o], q[0][3][o]),
                                   pack2(q[1][2][o], q[1][3][o]));
            }
        }
        __syncthreads();
        const T* B = static_cast<const T*>(a.b) + static_cast<long long>(t.e) * a.N * a.r;
        for (int n0 = c0 + 32 * w; n0 < c1; n0 += 32 * WARPS) {
            const int col = n0 + 8 * ti, cols = min(8, c1 - col);
            float acc[MT][4][4] = {};
            float add[MT][2][8];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = srow[16 * m + 8 * h + gi];
                    const bool there = base != nullptr && row >= 0 && cols > 0;
                    const O* p = base + row * a.base_stride + col;
                    if constexpr (VEC) {
                        constexpr int W = 16 / sizeof(O);
#pragma unroll
                        for (int i = 0; i < 8; i += W) {
                            Raw<O, W> v;
                            v.clear();
                            if (there) v.v = *reinterpret_cast<const uint4*>(p + i);
                            float f[W];
                            v.get(f);
#pragma unroll
                            for (int q = 0; q < W; ++q) add[m][h][i + q] = f[q];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) add[m][h][i] = there && i < cols ? to_f32(p[i]) : 0.0f;
                    }
                }
            if (adapted) {
                for (int ks = 0; ks < KS; ++ks) {
                    const int k = 16 * ks + 4 * ti;
                    uint2 fb[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int n = n0 + 8 * (gi >> 1) + 2 * j + (gi & 1);
                        fb[j] = load4<T, VEC>(B + static_cast<long long>(n) * a.r + k, n < c1 ? a.r - k : 0);
                    }
#pragma unroll
                    for (int o = 0; o < NP; ++o)
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint4 f = frag[((ks * NP + o) * MT + m) * 32 + lane];
#pragma unroll
                            for (int j = 0; j < 4; ++j) mma16816<T>(acc[m][j], f.x, f.y, f.z, f.w, fb[j].x, fb[j].y);
                        }
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = 16 * m + 8 * h + gi, row = srow[p];
                    if (row < 0 || cols <= 0) continue;
                    float f[8];
                    const float back = SCALED && adapted ? 1.0f / sscale[p] : 1.0f;  // a power of two
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = fmaf(acc[m][i >> 1][2 * h + (i & 1)], back, add[m][h][i]);
                    O* o = out + row * a.out_stride + col;
                    if constexpr (VEC) {
                        constexpr int W = 16 / sizeof(O);
#pragma unroll
                        for (int i = 0; i < 8; i += W) {
                            float e[W];
#pragma unroll
                            for (int q = 0; q < W; ++q) e[q] = f[i + q];
                            Raw<O, W> v;
                            v.set(e);
                            v.store(o + i);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i < cols) o[i] = from_f32<O>(f[i]);
                    }
                }
        }
    }
}

// Tiles of tm positions at most: a part full one a group, or a position each.
long long most_tiles(const AdapterArgs& a, int tm) {
    const long long part = a.E + 1 < a.T ? a.E + 1 : a.T;
    return (a.T + tm - 1) / tm + part;
}

template <typename K>
cudaError_t launch_units(K kernel, long long units, int per_sm, size_t smem, cudaStream_t s, const AdapterArgs& a) {
    const long long cap = static_cast<long long>(num_sms()) * per_sm;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(units < cap ? units : cap)), dim3(THREADS), smem, s, a);
}

template <typename T, typename O>
cudaError_t launch_simt(const AdapterArgs& a, cudaStream_t s) {
    cudaError_t e = launch_units(adapter_shrink_kernel<T>, most_tiles(a, SH_TILE) * ((a.r + SH_RANKS - 1) / SH_RANKS), 8, 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_units(adapter_expand_kernel<T, O>, most_tiles(a, EX_TILE) * ((a.N + THREADS - 1) / THREADS), 8, 0, s, a);
}

template <typename T, int MT, bool VEC>
cudaError_t shrink_mma(const AdapterArgs& a, cudaStream_t s) {
    const long long tiles = most_tiles(a, 16 * MT) * a.slices;
    if (a.rp <= 16) return launch_units(adapter_shrink_mma_kernel<T, MT, 2, VEC>, tiles, 4, 0, s, a);
    if (a.rp <= 32) return launch_units(adapter_shrink_mma_kernel<T, MT, 4, VEC>, tiles, 4, 0, s, a);
    return launch_units(adapter_shrink_mma_kernel<T, MT, 8, VEC>, tiles * ((a.rp + 63) / 64), 4, 0, s, a);
}

template <typename T, typename O, int MT, bool VEC>
cudaError_t expand_mma(AdapterArgs a, cudaStream_t s) {
    const long long tiles = most_tiles(a, 16 * MT);
    // a range of columns a CTA: 256 (one turn of its warps) while the CTAs are few, else up to 1024
    a.col_parts = static_cast<int>(std::max<long long>(1, std::min<long long>((a.N + 255) / 256, (8LL * num_sms() + tiles - 1) / tiles)));
    constexpr int STEP = (sizeof(O) == 4 ? 3 : 2) * MT * 512;  // of 16 ranks
    static bool done[64] = {};
    if (!allow_smem(adapter_expand_mma_kernel<T, O, MT, VEC>, 16 * STEP, done)) return cudaErrorInvalidValue;
    const size_t smem = static_cast<size_t>(a.rp / 16) * STEP;
    return launch_units(adapter_expand_mma_kernel<T, O, MT, VEC>, tiles * a.col_parts, 4, smem, s, a);
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <typename T, typename O>
cudaError_t launch_mma(const AdapterArgs& a, cudaStream_t s) {
    const bool in = a.d % 8 == 0 && a.x_stride % 8 == 0 && aligned_to(a.x, 16) && aligned_to(a.a, 16);
    const bool out = a.N % 8 == 0 && a.r % 4 == 0 && aligned_to(a.b, 8) && aligned_to(a.out, 16) &&
                     a.out_stride * sizeof(O) % 16 == 0 && aligned_to(a.base, 16) && a.base_stride * sizeof(O) % 16 == 0;
    const bool many = a.T >= 24LL * (a.E + 1);
    cudaError_t e;
    if (many) e = in ? shrink_mma<T, 2, true>(a, s) : shrink_mma<T, 2, false>(a, s);
    else e = in ? shrink_mma<T, 1, true>(a, s) : shrink_mma<T, 1, false>(a, s);
    if (e != cudaSuccess) return e;
    if (many) return out ? expand_mma<T, O, 2, true>(a, s) : expand_mma<T, O, 2, false>(a, s);
    return out ? expand_mma<T, O, 1, true>(a, s) : expand_mma<T, O, 1, false>(a, s);
}

// Slices of d: enough for two CTAs an SM, of 512 at least.
int adapter_slices(int T, int d, int E) {
    const long long tiles = (T + 31) / 32 + std::min<long long>(E, T);
    return static_cast<int>(std::max<long long>(1, std::min<long long>({(2LL * num_sms() + tiles - 1) / tiles, d / 512, 8})));
}

}  // namespace

size_t adapter_workspace(int T, int d, int r, int E, int dtype) {
    if (dtype == MOE_F32) return 256 + static_cast<size_t>(T) * r * 4;
    return 256 + static_cast<size_t>(T) * ((r + 15) / 16 * 16) * 4 * adapter_slices(T, d, E);
}

cudaError_t launch_adapter(const AdapterArgs& args, cudaStream_t s) {
    AdapterArgs a = args;
    if (a.dtype == MOE_F32) return launch_simt<float, float>(a, s);
    a.rp = (a.r + 15) / 16 * 16;
    a.slices = adapter_slices(a.T, a.d, a.E);
    const bool wide = a.out_dtype == MOE_F32;
    if (a.dtype == MOE_BF16) return wide ? launch_mma<__nv_bfloat16, float>(a, s) : launch_mma<__nv_bfloat16, __nv_bfloat16>(a, s);
    return wide ? launch_mma<__half, float>(a, s) : launch_mma<__half, __half>(a, s);
}

}  // namespace moe
