// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + s_e (x[t] A_e^T) B_e^T,   e the adapter of row t
//
// Rows come grouped by adapter: group e is the positions offsets[e] to offsets[e + 1]
// of `rows`; positions from offsets[E] on have no adapter. Two launches: the first
// computes v = s_e x[t] A_e^T into the workspace (by position, FP32), the second adds
// v B_e^T to base.
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

template <typename K>
cudaError_t launch_units(K kernel, long long units, cudaStream_t s, const AdapterArgs& a) {
    const long long cap = static_cast<long long>(num_sms()) * 8;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(units < cap ? units : cap)), dim3(THREADS), 0, s, a);
}

// Tiles of tm positions at most: a part full one a group, or a position each.
long long most_tiles(const AdapterArgs& a, int tm) {
    const long long part = a.E + 1 < a.T ? a.E + 1 : a.T;
    return (a.T + tm - 1) / tm + part;
}

template <typename T, typename O>
cudaError_t launch_t(const AdapterArgs& a, cudaStream_t s) {
    cudaError_t e = launch_units(adapter_shrink_kernel<T>, most_tiles(a, SH_TILE) * ((a.r + SH_RANKS - 1) / SH_RANKS), s, a);
    if (e != cudaSuccess) return e;
    return launch_units(adapter_expand_kernel<T, O>, most_tiles(a, EX_TILE) * ((a.N + THREADS - 1) / THREADS), s, a);
}

}  // namespace

size_t adapter_workspace(int T, int r) { return 256 + static_cast<size_t>(T) * r * 4; }

cudaError_t launch_adapter(const AdapterArgs& a, cudaStream_t s) {
    const bool wide = a.out_dtype == MOE_F32;
    switch (a.dtype) {
        case MOE_BF16: return wide ? launch_t<__nv_bfloat16, float>(a, s) : launch_t<__nv_bfloat16, __nv_bfloat16>(a, s);
        case MOE_F16: return wide ? launch_t<__half, float>(a, s) : launch_t<__half, __half>(a, s);
        default: return launch_t<float, float>(a, s);
    }
}

}  // namespace moe
