// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + s_e (x[t] A_e^T) B_e^T,   e the adapter of row t
//
// Rows come grouped by adapter: group e is the positions offsets[e] to offsets[e + 1]
// of `rows`; positions from offsets[E] on have no adapter. Three forms:
//   FP32: two launches, the first leaves the inner values v = s_e x[t] A_e^T in the workspace
//     (FP32, by position), the second adds v B_e^T to base.
//   16-bit types, few rows: one launch; v stays in shared memory.
//   16-bit types, many rows (adapter_tc.cu): two launches, v in pieces of the operands' type
//     in the workspace.
#include <stdlib.h>

#include "adapter.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// FP32
// ---------------------------------------------------------------------------
// v = s x A^T of 4 positions by 8 ranks and one slice of d, by a warp: its lanes take
// neighbouring elements of d, and the 32 sums are scattered over the lanes as they are added.
constexpr int F32_ROWS = 4, F32_RANKS = 8;

template <bool VEC>
__global__ void __launch_bounds__(THREADS, 2) adapter_shrink_f32_kernel(const __grid_constant__ AdapterArgs a) {
    constexpr int W = VEC ? 4 : 1;  // elements a lane loads at once
    __shared__ Groups g;
    pdl_wait();
    pdl_trigger();
    const int tiles = group_table<F32_ROWS>(a, false, g);
    const int lane = static_cast<int>(lane_id());
    const int rb = (a.rp + F32_RANKS - 1) / F32_RANKS, parts = rb * a.slices;
    const int len = ((a.d + a.slices - 1) / a.slices + 31) / 32 * 32;
    const float* x = static_cast<const float*>(a.x);
    const long long units = static_cast<long long>(tiles) * parts, step = static_cast<long long>(gridDim.x) * (THREADS / 32);
    for (long long u = static_cast<long long>(threadIdx.x >> 5) * gridDim.x + blockIdx.x; u < units; u += step) {
        const Tile t = tile_of<F32_ROWS>(static_cast<int>(u / parts), a, g);
        const int part = static_cast<int>(u % parts), j0 = part % rb * F32_RANKS, slice = part / rb;
        const int k0 = slice * len, k1 = min(a.d, k0 + len);
        const float* xr[F32_ROWS];
#pragma unroll
        for (int i = 0; i < F32_ROWS; ++i) {
            const int r = i < t.n ? row_of(a, t.pos + i) : 0;
            if (r < 0 && lane == 0) atomicOr(a.err, ERRBIT_INDEX);
            xr[i] = x + max(r, 0) * a.x_stride;
        }
        const float* A = static_cast<const float*>(a.a) + (static_cast<long long>(t.e) * a.r + j0) * a.d;
        float acc[F32_ROWS * F32_RANKS] = {};
#pragma unroll 2
        for (int k = k0 + lane * W; k < k1; k += 32 * W) {
            float xv[F32_ROWS][W], av[F32_RANKS][W];
#pragma unroll
            for (int i = 0; i < F32_ROWS; ++i) load_f32<W>(xr[i] + k, xv[i]);
#pragma unroll
            for (int j = 0; j < F32_RANKS; ++j) {
                // ranks behind r read the last one, and are not stored
                load_f32<W>(A + static_cast<long long>(min(j, a.r - 1 - j0)) * a.d + k, av[j]);
            }
#pragma unroll
            for (int i = 0; i < F32_ROWS; ++i)
#pragma unroll
                for (int j = 0; j < F32_RANKS; ++j)
#pragma unroll
                    for (int q = 0; q < W; ++q) acc[i * F32_RANKS + j] = fmaf(xv[i][q], av[j][q], acc[i * F32_RANKS + j]);
        }
        // each turn halves the sums a lane holds: lane l ends with sum l
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < o; ++i) {
                const float keep = up ? acc[i + o] : acc[i], give = up ? acc[i] : acc[i + o];
                acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        }
        const int p = lane / F32_RANKS, rank = j0 + lane % F32_RANKS;
        const float s = a.scale != nullptr ? __ldg(a.scale + t.e) : 1.0f;
        if (p < t.n && rank < a.rp)
            a.v[(static_cast<long long>(slice) * a.T + t.pos + p) * a.rp + rank] = rank < a.r ? s * acc[0] : 0.0f;
    }
}

// out = base + v B^T of 64 positions by ranges of 128 columns, 32 ranks at a time through shared
// memory (the next ones in registers meanwhile): a warp has 8 rows, a lane 4 columns of each. B is
// turned around on its way in; element (j, n) lies at n ^ 4 (j / 4), so that neither the
// writes nor the 16-byte reads meet in a bank.
constexpr int F32_TILE = 64, F32_COLS = 128, F32_STEP = 32;

template <bool VEC>
__global__ void __launch_bounds__(THREADS, 2) adapter_expand_f32_kernel(const __grid_constant__ AdapterArgs a) {
    constexpr int PER = F32_TILE / (THREADS / 32), BN = F32_COLS * F32_STEP / 4 / THREADS, VN = F32_TILE * F32_STEP / 4 / THREADS;
    __shared__ Groups g;
    __shared__ __align__(16) float sv[F32_TILE][F32_STEP], sb[F32_STEP][F32_COLS];
    __shared__ int srow[F32_TILE];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int nb = a.col_parts, len = ((a.N + nb - 1) / nb + F32_COLS - 1) / F32_COLS * F32_COLS;
    const float* base = static_cast<const float*>(a.base);
    float* out = static_cast<float*>(a.out);
    const bool bvec = a.r % 4 == 0 && reinterpret_cast<uintptr_t>(a.b) % 16 == 0;
    // ranks of a step in fours, rounded up to a power of two
    const int quads = a.rp > 16 ? 8 : a.rp > 8 ? 4 : a.rp > 4 ? 2 : 1, ql = a.rp > 16 ? 3 : a.rp > 8 ? 2 : a.rp > 4 ? 1 : 0;
    pdl_wait();
    pdl_trigger();
    const int tiles = group_table<F32_TILE>(a, !a.in_place, g);
    for (long long u = blockIdx.x; u < static_cast<long long>(tiles) * nb; u += gridDim.x) {
        const Tile t = tile_of<F32_TILE>(static_cast<int>(u / nb), a, g);
        const int c0 = static_cast<int>(u % nb) * len, c1 = min(a.N, c0 + len);
        const int ranks = t.e < a.E ? a.rp : 0;
        const float* B = static_cast<const float*>(a.b) + static_cast<long long>(t.e) * a.N * a.r;
        __syncthreads();
        if (tid < F32_TILE) {
            srow[tid] = tid < t.n ? row_of(a, t.pos + tid) : -1;
            if (ranks == 0 && c0 == 0 && tid < t.n && srow[tid] < 0) atomicOr(a.err, ERRBIT_INDEX);  // the others': the first launch
        }
        // four ranks of a column (of a row of v) by neighbouring threads
        float4 bv[BN], vv[VN];
        auto fetch = [&](int n0, int j0) {
#pragma unroll
            for (int i = 0; i < BN; ++i) {
                const int at = tid + THREADS * i, n = n0 + (at >> ql), j = j0 + (at & (quads - 1)) * 4;
                bv[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (at >= F32_COLS * quads || n >= c1 || j >= a.r) continue;
                const float* p = B + static_cast<long long>(n) * a.r + j;
                if (bvec) {
                    bv[i] = __ldg(reinterpret_cast<const float4*>(p));
                } else {
                    bv[i].x = __ldg(p);
                    if (j + 1 < a.r) bv[i].y = __ldg(p + 1);
                    if (j + 2 < a.r) bv[i].z = __ldg(p + 2);
                    if (j + 3 < a.r) bv[i].w = __ldg(p + 3);
                }
            }
            if (n0 != c0 && ranks <= F32_STEP) return;  // v is there
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const int at = tid + THREADS * i, r = (at >> ql), j = j0 + (at & (quads - 1)) * 4;
                vv[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (at < F32_TILE * quads && r < t.n && j < a.rp) vv[i] = inner4(a, t.pos + r, j, a.slices);
            }
        };
        if (ranks > 0) fetch(c0, 0);
        __syncthreads();
        int row[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) row[i] = srow[w * PER + i];
        auto column = [&](int i) { return VEC ? 4 * lane + i : lane + 32 * i; };  // of a range, the lane's i-th
        for (int n0 = c0; n0 < c1; n0 += F32_COLS) {
            float acc[PER][4] = {};
            for (int j0 = 0; j0 < ranks; j0 += F32_STEP) {
                __syncthreads();  // the last step has been read
#pragma unroll
                for (int i = 0; i < BN; ++i) {
                    const int at = tid + THREADS * i, n = (at >> ql), j = (at & (quads - 1)) * 4, to = n ^ j;
                    if (at >= F32_COLS * quads) continue;
                    sb[j][to] = bv[i].x;
                    sb[j + 1][to] = bv[i].y;
                    sb[j + 2][to] = bv[i].z;
                    sb[j + 3][to] = bv[i].w;
                }
                if (n0 == c0 || ranks > F32_STEP) {
#pragma unroll
                    for (int i = 0; i < VN; ++i) {
                        const int at = tid + THREADS * i;
                        if (at < F32_TILE * quads) *reinterpret_cast<float4*>(&sv[(at >> ql)][(at & (quads - 1)) * 4]) = vv[i];
                    }
                }
                __syncthreads();
                if (j0 + F32_STEP < ranks) fetch(n0, j0 + F32_STEP);
                else if (n0 + F32_COLS < c1) fetch(n0 + F32_COLS, 0);
                const int steps = min(F32_STEP, ranks - j0);
                for (int j = 0; j < steps; j += 4) {
                    float b[4][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if constexpr (VEC) {
                            const float4 v = *reinterpret_cast<const float4*>(&sb[j + q][(4 * lane) ^ j]);
                            b[q][0] = v.x; b[q][1] = v.y; b[q][2] = v.z; b[q][3] = v.w;
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) b[q][i] = sb[j + q][column(i) ^ j];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const float4 v = *reinterpret_cast<const float4*>(&sv[w * PER + i][j]);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[i][q] = fmaf(v.w, b[3][q], fmaf(v.z, b[2][q], fmaf(v.y, b[1][q], fmaf(v.x, b[0][q], acc[i][q]))));
                    }
                }
            }
            float add[PER][4];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const bool there = base != nullptr && row[i] >= 0;
                const float* p = base + row[i] * a.base_stride + n0;
                if constexpr (VEC) {  // base may be out: no read-only loads
                    const float4 v = there && n0 + column(0) < c1 ? *reinterpret_cast<const float4*>(p + column(0)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    add[i][0] = v.x; add[i][1] = v.y; add[i][2] = v.z; add[i][3] = v.w;
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) add[i][q] = there && n0 + column(q) < c1 ? p[column(q)] : 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (row[i] < 0) continue;
                float* o = out + row[i] * a.out_stride + n0;
                if constexpr (VEC) {
                    if (n0 + column(0) < c1)
                        *reinterpret_cast<float4*>(o + column(0)) =
                            make_float4(add[i][0] + acc[i][0], add[i][1] + acc[i][1], add[i][2] + acc[i][2], add[i][3] + acc[i][3]);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (n0 + column(q) < c1) o[column(q)] = add[i][q] + acc[i][q];
                }
            }
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

// The 16 bytes at p of a 32-byte window [lo, hi] that begins s < 16 bytes before p.
MOE_DEV uint4 window(uint4 lo, uint4 hi, uint32_t s) {
    uint32_t w[7] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z};
    const uint32_t last = hi.w;
    if (s & 8) {
        w[0] = w[2]; w[1] = w[3]; w[2] = w[4]; w[3] = w[5]; w[4] = w[6]; w[5] = last;
    }
    if (s & 4) {
        w[0] = w[1]; w[1] = w[2]; w[2] = w[3]; w[3] = w[4]; w[4] = w[5];
    }
    if (s & 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 elements from p, zeros from the n-th on; `before` elements of the row lie in front of p. Two
// aligned loads where both lie within the row.
template <typename T>
MOE_DEV uint4 load8(const T* p, int before, int n) {
    const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
    if (s == 0 ? n >= 8 : before >= 8 && n >= 16) {
        const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - s);
        const uint4 lo = __ldg(q);
        return s == 0 ? lo : window(lo, __ldg(q + 1), s);
    }
    uint32_t w[4] = {0, 0, 0, 0};
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) w[i / 2] |= static_cast<uint32_t>(__ldg(q + i)) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// 4 elements from p, zeros from the n-th on; vec: 8-byte aligned, n a multiple of 4.
template <typename T>
MOE_DEV uint2 load4(const T* p, int n, bool vec) {
    if (vec) return n > 0 ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
    uint32_t w[2] = {0, 0};
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) w[i / 2] |= static_cast<uint32_t>(__ldg(q + i)) << (16 * (i & 1));
    return make_uint2(w[0], w[1]);
}

MOE_DEV void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Both products of a tile of 16 MT positions by a cluster of C CTAs, in one launch.
//   v: CTA c takes the c-th part of d, its warps every eighth 32 of that, 8 NT ranks a pass;
//   the warps' sums are added in order through shared memory, then the CTAs' in order through
//   the cluster's. base is on its way to L2 meanwhile (B with it would take the rate from A: 256
//   rows, 4096 x 4096, rank 16, 22.6 us for 20.7).
//   out: CTA c takes the c-th part of N, a warp 32 columns at a time. Column 2 i + q of its
//   instruction j stands for column 8 i + 2 j + q, so that a lane ends with 8 consecutive
//   columns of its rows.
// KB: steps of 16 ranks whose B is taken at once, the next ones under way. From two steps on a
// lane's ranks are 8 consecutive ones of 32 (rp a multiple of 16 KB), else 4 of 16.
// Every CTA makes the same number of turns, whatever the offsets: cluster barriers always pair.
template <typename T, typename O, int MT, int NT, int KB, bool VEC>
struct Fused {
    static constexpr int WARPS = THREADS / 32, ROWS = 16 * MT;
    static constexpr int NP = sizeof(O) == 4 ? 3 : 2;
    // Chunks of 32 of d a warp has in flight: on their way to shared memory, each lane's fragments to
    // its own 16-byte slots (two CTAs an SM leave 72 KB each; ranks past 64 take more for v and its
    // pieces, see ctas_an_sm), or, where rows are on no 16 bytes, to registers.
    static constexpr int FRAGS = 2 * MT + NT, U = FRAGS <= 4 ? 4 : FRAGS <= 6 ? 3 : 2;
    static constexpr int RING = VEC ? WARPS * U * FRAGS * 512 : 0;
    // The same slots then take B: steps under way, of 16-byte slots each.
    static constexpr int B_SLOTS = KB == 1 ? 2 : 2 * KB, B_STEPS = U * FRAGS / B_SLOTS < 8 ? U * FRAGS / B_SLOTS : 8;
    static constexpr int STAGE_OUT = VEC ? 0 : WARPS * 16 * 33 * 4;
    static constexpr int RED0 = WARPS * NT * 512, RED = RED0 > STAGE_OUT ? RED0 : STAGE_OUT;
    static size_t smem(int rp) {  // [part][red, then the sums and the columns on their way out][pieces][slots]
        const int sums = ROWS * rp * 4;
        return static_cast<size_t>(sums) + (RED > sums ? RED : sums) + static_cast<size_t>(rp / 16) * NP * MT * 512 + RING;
    }
    static constexpr int MOST = ROWS * 256 * 4 + (RED > ROWS * 1024 ? RED : ROWS * 1024) + 16 * NP * MT * 512 + RING;
    static_assert(MOST <= 220 << 10, "shared memory");
};
template <typename T, typename O, int MT, int NT, int KB, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) adapter_mma_kernel(const __grid_constant__ AdapterArgs a, int turns) {
    using F = Fused<T, O, MT, NT, KB, VEC>;
    constexpr int WARPS = F::WARPS, ROWS = F::ROWS, NP = F::NP, U = F::U;
    constexpr bool SCALED = __is_same(T, __half);
    constexpr int STEP = 32 * WARPS;
    // FP32 outputs of more than 16 ranks: the small pieces of v are summed apart, since what an addition
    // drops grows with the sum (in one accumulator, 256 rows of 128, rank 64: 2.7e-7 off for 1.9e-7)
    constexpr bool APART = sizeof(O) == 4 && NT > 2;
    // the next columns' base too: where B and the sums take few registers (32 rows and two accumulators: 2000 rows
    // of 8, 1024 x 4096, rank 28, 37 us with it, 29 without)
    constexpr bool AHEAD = VEC && KB == 1 && !(APART && MT == 2);
    __shared__ Groups g;
    __shared__ int srow[ROWS];
    __shared__ float sscale[SCALED ? ROWS : 1], sback[SCALED ? ROWS : 1];
    extern __shared__ __align__(16) uint8_t smem[];
    const int rp = a.rp, KS = rp / 16, C = a.cluster;
    float* part = reinterpret_cast<float*>(smem);  // [ROWS][rp], this CTA's part of d
    float* red = part + ROWS * rp;                 // [WARPS][NT * 4][32], then [ROWS][rp]
    uint4* frag = reinterpret_cast<uint4*>(red + (F::RED / 4 > ROWS * rp ? F::RED / 4 : ROWS * rp));  // [KS][NP][MT][32]
    uint4* slots = frag + KS * NP * MT * 32 + (threadIdx.x >> 5) * (F::RING / WARPS / 16) + (threadIdx.x & 31);  // this lane's, 32 apart
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, gi = lane >> 2, ti = lane & 3;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int clusters = gridDim.x / C, id = blockIdx.x / C;
    pdl_wait();
    pdl_trigger();
    const int tiles = group_table<ROWS>(a, !a.in_place, g);
    const int klen = ((a.d + C - 1) / C + 31) / 32 * 32, nlen = ((a.N + C - 1) / C + 31) / 32 * 32;
    const int k0 = min(a.d, rank * klen), k1 = min(a.d, k0 + klen), c0 = min(a.N, rank * nlen), c1 = min(a.N, c0 + nlen);
    const T* x = static_cast<const T*>(a.x);
    const O* base = static_cast<const O*>(a.base);
    O* out = static_cast<O*>(a.out);
    const bool bvec = a.r % 4 == 0 && reinterpret_cast<uintptr_t>(a.b) % 8 == 0;
    for (int turn = 0; turn < turns; ++turn) {
        const int tile = turn * clusters + id;
        Tile t{a.E, 0, 0};
        if (tile < tiles) t = tile_of<ROWS>(tile, a, g);
        const bool adapted = t.e < a.E;
        const T* B = static_cast<const T*>(a.b) + static_cast<long long>(t.e) * a.N * a.r;
        __syncthreads();  // the last turn's rows have been read
        if (tid < ROWS) {
            srow[tid] = tid < t.n ? row_of(a, t.pos + tid) : -1;
            if (tid < t.n && srow[tid] < 0 && rank == 0) atomicOr(a.err, ERRBIT_INDEX);
        }
        __syncthreads();
        if (base != nullptr && c1 > c0) {
            const int lines = ((c1 - c0) * static_cast<int>(sizeof(O)) + 127) / 128;
            for (int i = tid; i < t.n * lines; i += THREADS) {
                const int row = srow[i / lines];
                if (row >= 0) prefetch_l2(reinterpret_cast<const char*>(base + row * a.base_stride + c0) + i % lines * 128);
            }
        }
        if (adapted) {
            int row[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) row[m][h] = srow[16 * m + 8 * h + gi];
            const int first = k0 + 32 * w, chunks = first < k1 ? (k1 - first + 32 * WARPS - 1) / (32 * WARPS) : 0;
            const int passes = (rp + 8 * NT - 1) / (8 * NT);
            // VEC: chunk after chunk, pass after pass, on their way to the slots
            int ip = 0, iq = 0, is = 0;
            auto issue = [&] {
                if (ip < passes && iq < chunks) {
                    const int at = first + 32 * WARPS * iq + 8 * ti;
                    uint4* slot = slots + is * F::FRAGS * 32;
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (16 * m + 8 * h < t.n)  // else what is there goes into rows that nobody reads
                                cp_async_16z(smem_u32(slot + (2 * m + h) * 32), x + max(row[m][h], 0) * a.x_stride + at,
                                             row[m][h] >= 0 && at < k1);
                    const int rank0 = 8 * NT * ip + gi;
                    const T* A = static_cast<const T*>(a.a) + (static_cast<long long>(t.e) * a.r + rank0) * a.d + at;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        cp_async_16z(smem_u32(slot + (2 * MT + j) * 32), rank0 + 8 * j < a.r ? A + static_cast<long long>(8 * j) * a.d : x,
                                     rank0 + 8 * j < a.r && at < k1);
                    if (++iq == chunks) {
                        iq = 0;
                        ++ip;
                    }
                }
                if (++is == U) is = 0;
                cp_async_commit();
            };
            int slot_at = 0;
            if constexpr (VEC) {
#pragma unroll
                for (int c = 0; c < U; ++c) issue();
            }
            for (int j0 = 0; j0 < rp; j0 += 8 * NT) {
                float acc[MT][NT][4] = {};
                auto multiply = [&](const uint4 (&fx)[MT][2], const uint4 (&fa)[NT]) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            mma16816<T>(acc[m][j], fx[m][0].x, fx[m][1].x, fx[m][0].y, fx[m][1].y, fa[j].x, fa[j].y);
                            mma16816<T>(acc[m][j], fx[m][0].z, fx[m][1].z, fx[m][0].w, fx[m][1].w, fa[j].z, fa[j].w);
                        }
                };
                if constexpr (VEC) {
                    for (int q = 0; q < chunks; ++q) {
                        cp_async_wait<U - 1>();
                        uint4 fx[MT][2], fa[NT];
                        const uint4* slot = slots + slot_at * F::FRAGS * 32;
#pragma unroll
                        for (int i = 0; i < 2 * MT; ++i) fx[i / 2][i & 1] = slot[i * 32];
#pragma unroll
                        for (int j = 0; j < NT; ++j) fa[j] = slot[(2 * MT + j) * 32];
                        if (++slot_at == U) slot_at = 0;
                        issue();  // into the slots just read, which are this lane's alone
                        multiply(fx, fa);
                    }
                } else {
                    const T* A = static_cast<const T*>(a.a) + (static_cast<long long>(t.e) * a.r + j0 + gi) * a.d;
                    uint4 fx[U][MT][2], fa[U][NT];
                    auto load = [&](int c, int k) {
                        const int at = k + 8 * ti, n = k1 - at;
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                fx[c][m][h] = load8<T>(x + max(row[m][h], 0) * a.x_stride + at, at, row[m][h] >= 0 ? n : 0);
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            fa[c][j] = load8<T>(A + static_cast<long long>(8 * j) * a.d + at, at, j0 + 8 * j + gi < a.r ? n : 0);
                    };
#pragma unroll
                    for (int c = 0; c < U; ++c) load(c, first + 32 * WARPS * c);
                    for (int k = first; k < k1; k += 32 * WARPS * U) {
#pragma unroll
                        for (int c = 0; c < U; ++c) {
                            multiply(fx[c], fa[c]);  // chunks behind the part are zeros
                            load(c, k + 32 * WARPS * (c + U));
                        }
                    }
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) red[(w * NT + j) * 128 + 32 * i + lane] = acc[m][j][i];
                    __syncthreads();
                    for (int i = tid; i < NT * 128; i += THREADS) {
                        float v = red[i];
#pragma unroll
                        for (int o = 1; o < WARPS; ++o) v += red[o * NT * 128 + i];
                        const int l = i & 31, q = i >> 5 & 3, j = i / 128;
                        const int col = j0 + 8 * j + 2 * (l & 3) + (q & 1);
                        if (col < rp) part[(16 * m + 8 * (q >> 1) + (l >> 2)) * rp + col] = v;
                    }
                    __syncthreads();
                }
            }
        }
        // B of a step (32 columns, 16 KB ranks) by this lane, and for VEC the first ones under way
        // while the parts meet.
        const int nsteps = (KS + KB - 1) / KB;
        const int blocks = adapted && c0 + 32 * w < c1 ? (c1 - c0 - 32 * w + STEP - 1) / STEP : 0;
        int bn = 0, bk = 0, bs = 0;
        auto issue_b = [&] {
            if (bn < blocks) {
                const int n0 = c0 + 32 * w + STEP * bn;
                uint4* slot = slots + bs * F::B_SLOTS * 32;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = n0 + 8 * (gi >> 1) + 2 * j + (gi & 1);
                    const T* p = B + static_cast<long long>(n) * a.r;
                    if constexpr (KB == 1) {
                        const int k = 16 * bk + 4 * ti;
                        const bool there = n < c1 && k < a.r;
                        cp_async_8z(smem_u32(slot + j / 2 * 32) + 8 * (j & 1), there ? p + k : B, there);
                    } else {
#pragma unroll
                        for (int q = 0; q < KB; q += 2) {
                            const int k = 16 * (KB * bk + q) + 8 * ti;
                            const bool there = n < c1 && k < a.r;
                            cp_async_16z(smem_u32(slot + (j * KB / 2 + q / 2) * 32), there ? p + k : B, there);
                        }
                    }
                }
                if (++bk == nsteps) {
                    bk = 0;
                    ++bn;
                }
            }
            if (++bs == F::B_STEPS) bs = 0;
            cp_async_commit();
        };
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < F::B_STEPS; ++i) issue_b();
        }
        if (C > 1) cluster_sync();  // all parts of d are there
        if (adapted) {
            const float s = a.scale != nullptr ? __ldg(a.scale + t.e) : 1.0f;
            for (int i = tid; i < ROWS * rp / 4; i += THREADS) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (C > 1) {
                    const uint32_t at = smem_u32(part + 4 * i);
#pragma unroll 4
                    for (int c = 0; c < C; ++c) {
                        const float4 o = ld_shared_cluster_v4(map_shared_rank(at, c));
                        v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
                    }
                } else {
                    v = *reinterpret_cast<const float4*>(part + 4 * i);
                }
                const int k = 4 * i % rp;  // ranks behind r are zeros whatever x holds
                v.x = k < a.r ? v.x * s : 0.0f;
                v.y = k + 1 < a.r ? v.y * s : 0.0f;
                v.z = k + 2 < a.r ? v.z * s : 0.0f;
                v.w = k + 3 < a.r ? v.w * s : 0.0f;
                *reinterpret_cast<float4*>(red + 4 * i) = v;
            }
        }
        if (C > 1) cluster_arrive();  // the others' parts have been read
        __syncthreads();
        if (adapted) {
            if constexpr (SCALED) {
                constexpr int PER = THREADS / ROWS;  // threads a row, within a warp
                const int p = tid / PER;
                float most = 0.0f;
                for (int k = tid % PER * 4; k < rp; k += PER * 4) most = largest_finite(*reinterpret_cast<const float4*>(red + p * rp + k), most);
#pragma unroll
                for (int o = PER / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                if (tid % PER == 0) row_scale(most, sscale[p], sback[p]);
                __syncthreads();
            }
            for (int i = tid; i < KS * MT * 32; i += THREADS) {
                const int l = i & 31, m = i / 32 % MT, ks = i / (32 * MT);
                const int k = KB == 1 ? 16 * ks + 4 * (l & 3) : 32 * (ks >> 1) + 8 * (l & 3) + 4 * (ks & 1);
                T q[2][4][NP];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = 16 * m + 8 * h + (l >> 2);
                    const float4 v = *reinterpret_cast<const float4*>(red + p * rp + k);
                    const float f = SCALED ? sscale[p] : 1.0f;
                    split<T, NP>(v.x * f, q[h][0]);
                    split<T, NP>(v.y * f, q[h][1]);
                    split<T, NP>(v.z * f, q[h][2]);
                    split<T, NP>(v.w * f, q[h][3]);
                }
#pragma unroll
                for (int o = 0; o < NP; ++o)
                    frag[((ks * NP + o) * MT + m) * 32 + l] =
                        make_uint4(pack2(q[0][0][o], q[0][1][o]), pack2(q[1][0][o], q[1][1][o]), pack2(q[0][2][o], q[0][3][o]),
                                   pack2(q[1][2][o], q[1][3][o]));
            }
            __syncthreads();
        }
        int row[MT][2];
        float back[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                row[m][h] = srow[16 * m + 8 * h + gi];
                back[m][h] = SCALED && adapted ? sback[16 * m + 8 * h + gi] : 1.0f;
            }
        Cols<O> add[MT][2];
        auto load_base = [&](int n0) {
            const int col = n0 + 8 * ti;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    add[m][h].load(base + row[m][h] * a.base_stride + col, base != nullptr && row[m][h] >= 0 && col < c1);
        };
        uint2 fb[4];  // !VEC: the next step's
        auto load_b = [&](int n0, int ks) {
            const int k = 16 * ks + 4 * ti;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + 8 * (gi >> 1) + 2 * j + (gi & 1);
                fb[j] = load4<T>(B + static_cast<long long>(n) * a.r + k, adapted && n < c1 ? a.r - k : 0, bvec);
            }
        };
        // rank k of row p from its pieces (FP16: times the row's scale)
        auto whole = [&](int p, int k) {
            const int ks = KB == 1 ? k / 16 : 2 * (k / 32) + (k >> 2 & 1), l = 4 * (p & 7) + (KB == 1 ? k >> 2 & 3 : k >> 3 & 3);
            float v = 0.0f;
#pragma unroll
            for (int o = 0; o < NP; ++o)
                v += to_f32(reinterpret_cast<const T*>(frag + ((ks * NP + o) * MT + (p >> 4)) * 32 + l)[(k >> 1 & 1) * 4 + (p >> 3 & 1) * 2 + (k & 1)]);
            return v;
        };
        int b_at = 0;
        if constexpr (!VEC) load_b(c0 + 32 * w, 0);
        if constexpr (AHEAD) load_base(c0 + 32 * w);
        for (int n0 = c0 + 32 * w; t.n > 0 && n0 < c1; n0 += STEP) {
            Cols<O> here[MT][2];
            if constexpr (AHEAD) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) here[m][h] = add[m][h];
                load_base(n0 + STEP);
            } else if constexpr (VEC) {
                load_base(n0);
            }
            float acc[MT][4][4] = {}, less[APART ? MT : 1][4][4] = {};
            for (int ks = 0; adapted && ks < KS; ks += KB) {
                uint2 cur[KB][4];
                if constexpr (VEC) {
                    cp_async_wait<F::B_STEPS - 1>();
                    const uint4* slot = slots + b_at * F::B_SLOTS * 32;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (KB == 1) {
                            cur[0][j] = reinterpret_cast<const uint2*>(slot + j / 2 * 32)[j & 1];
                        } else {
#pragma unroll
                            for (int q = 0; q < KB; q += 2) {
                                const uint4 v = slot[(j * KB / 2 + q / 2) * 32];
                                cur[q][j] = make_uint2(v.x, v.y);
                                cur[q + 1][j] = make_uint2(v.z, v.w);
                            }
                        }
                    }
                    if (++b_at == F::B_STEPS) b_at = 0;
                    issue_b();
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) cur[0][j] = fb[j];
                    if (ks + KB < KS) load_b(n0, ks + KB);
                    else load_b(n0 + STEP, 0);
                }
#pragma unroll
                for (int q = 0; q < KB; ++q)
#pragma unroll
                    for (int o = NP - 1; o >= 0; --o)
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint4 f = frag[(((ks + q) * NP + o) * MT + m) * 32 + lane];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma16816<T>(APART && o > 0 ? less[APART ? m : 0][j] : acc[m][j], f.x, f.y, f.z, f.w, cur[q][j].x, cur[q][j].y);
                        }
            }
            if constexpr (APART) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[m][j][i] += less[m][j][i];
            }
            if constexpr (VEC) {
                const int col = n0 + 8 * ti;
                uint32_t again = 0;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (row[m][h] < 0 || col >= c1) continue;
                        const Cols<O>& old = AHEAD ? here[m][h] : add[m][h];
                        O* to = out + row[m][h] * a.out_stride + col;
                        if (adapted) {
                            F2 v[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) v[j] = f2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
                            const bool nan = any_nan(v);
                            if (nan) again |= 1u << (2 * m + h);
                            else old.add_to(to, v, back[m][h]);
                        } else {
                            old.copy_to(to);
                        }
                    }
                if (again != 0) {
#pragma unroll 1
                    for (int i = 0; i < 2 * MT; ++i) {
                        if ((again >> i & 1) == 0) continue;
                        const int p = 8 * i + gi, at = srow[p];
                        store_again(out + at * a.out_stride + col, base != nullptr ? base + at * a.base_stride + col : nullptr,
                                    [&](int k) { return whole(p, k); }, B + static_cast<long long>(col) * a.r, a.r, SCALED ? sback[p] : 1.0f);
                    }
                }
            } else {
                // rows on no 16 bytes: 16 rows of the warp's columns through shared memory, then a row's
                // 32 columns by the 32 lanes
                float* mine = red + w * 16 * 33;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 8; ++i) mine[(8 * h + gi) * 33 + 8 * ti + i] = acc[m][i >> 1][2 * h + (i & 1)] * back[m][h];
                    uint32_t again = 0;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        F2 v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = f2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
                        if (any_nan(v) && row[m][h] >= 0) again |= 1u << h;
                    }
                    if (adapted && again != 0) {
                        const int at = n0 + 8 * ti;
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            if ((again >> h & 1) == 0) continue;
                            const int p = 16 * m + 8 * h + gi;
                            float s[8];
                            sums_again(s, [&](int k) { return whole(p, k); }, B + static_cast<long long>(at) * a.r, a.r, c1 - at);
#pragma unroll
                            for (int i = 0; i < 8; ++i) mine[(8 * h + gi) * 33 + 8 * ti + i] = s[i] * (SCALED ? sback[p] : 1.0f);
                        }
                    }
                    __syncwarp();
                    const int col = n0 + lane;
                    O old[16];
#pragma unroll
                    for (int p = 0; p < 16; ++p) {
                        const int r = srow[16 * m + p];
                        old[p] = base != nullptr && r >= 0 && col < c1 ? base[r * a.base_stride + col] : from_f32<O>(0.0f);
                    }
#pragma unroll
                    for (int p = 0; p < 16; ++p) {
                        const int r = srow[16 * m + p];
                        if (r >= 0 && col < c1) out[r * a.out_stride + col] = adapted ? from_f32<O>(to_f32(old[p]) + mine[p * 33 + lane]) : old[p];
                    }
                }
            }
        }
        if (C > 1) cluster_wait();
    }
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Tiles of tm positions at most: a part full one a group, or a position each.
long long most_tiles(const AdapterArgs& a, int tm) {
    return std::min<long long>(a.T, (a.T + tm - 1) / tm + a.E + 1);
}

template <typename K>
cudaError_t launch_units(K kernel, long long units, int per_sm, size_t smem, cudaStream_t s, const AdapterArgs& a) {
    const long long cap = static_cast<long long>(num_sms()) * per_sm;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(units < cap ? units : cap)), dim3(THREADS), smem, s, a);
}

cudaError_t launch_f32(AdapterArgs a, cudaStream_t s) {
    const bool in = a.d % 4 == 0 && a.x_stride % 4 == 0 && aligned_to(a.x, 16) && aligned_to(a.a, 16);
    const long long units = most_tiles(a, F32_ROWS) * ((a.rp + F32_RANKS - 1) / F32_RANKS) * a.slices;
    const cudaError_t e = launch_units(in ? adapter_shrink_f32_kernel<true> : adapter_shrink_f32_kernel<false>, units, 3, 0, s, a);
    if (e != cudaSuccess) return e;
    const bool out = a.N % 4 == 0 && aligned_to(a.out, 16) && a.out_stride % 4 == 0 && aligned_to(a.base, 16) && a.base_stride % 4 == 0;
    const long long tiles = most_tiles(a, F32_TILE);
    a.col_parts = static_cast<int>(std::max<long long>(1, std::min<long long>((a.N + F32_COLS - 1) / F32_COLS, (4LL * num_sms() + tiles - 1) / tiles)));
    return launch_units(out ? adapter_expand_f32_kernel<true> : adapter_expand_f32_kernel<false>, tiles * a.col_parts, 2, 0, s, a);
}

template <typename T, typename O, int MT, int NT, int KB, bool VEC>
cudaError_t fused_k(AdapterArgs a, cudaStream_t s) {
    using F = Fused<T, O, MT, NT, KB, VEC>;
    static bool done[64] = {};
    if (!allow_smem(adapter_mma_kernel<T, O, MT, NT, KB, VEC>, F::MOST, done)) return cudaErrorInvalidValue;
    const long long tiles = most_tiles(a, 16 * MT), per_sm = ctas_an_sm(F::smem(a.rp)), places = per_sm * num_sms();
    // As many CTAs a tile as there are places for, while each has 256 of d and of N; a tenth more
    // may wait, as tiles are counted for adapters that all have rows (256 rows of 64, 2048 x 8192,
    // rank 32: 4 CTAs 16 us, 2 CTAs 25; but twice the places, 256 of 128, 4096 x 4096, rank 64: 47 for 39).
    // Where an SM holds one (large ranks, 4096 x 4096) a third more, but no more than the places for clusters of
    // 8, which the SMs' groups have less room for (256 rows of 32, rank 128, FP32 output, 49 tiles counted and 32
    // there: 4 CTAs 25 us, 2 CTAs 39; 64 of 16: 8 CTAs 31 us, 4 CTAs 22; 256 of 16, rank 256: 8 CTAs 55, 4 CTAs 41).
    const long long most = per_sm == 2 ? places * 11 / 10 : places * 4 / 3;
    a.cluster = 1;
    while (a.cluster < 8 && tiles * a.cluster * 2 <= (per_sm == 1 && a.cluster == 4 ? places : most) && std::min(a.d, a.N) >= 512 * a.cluster)
        a.cluster *= 2;
    const long long clusters = tiles * a.cluster <= most ? tiles : places / a.cluster;
    const int turns = static_cast<int>((tiles + clusters - 1) / clusters);
    return launch_pdl_cluster(adapter_mma_kernel<T, O, MT, NT, KB, VEC>, dim3(static_cast<unsigned>(clusters * a.cluster)), dim3(THREADS),
                              F::smem(a.rp), s, a.cluster, a, turns);
}

// Whether a call of 16-bit types goes to the kernels of many rows, where its operands allow it:
// from a number of inner values on, and while adapters have 16 rows of rank 64 (64 of rank 16)
// each if all have any. (us, few rows' kernel : many rows', d and N 4096 unless given. 1024 rows
// of 8 adapters, rank 64, 31 : 24; rank 16, 17 : 18; 512 of 4, rank 128, 2048 x 2048, 30 : 19; 4096
// rows of 64, rank 64, 102 : 60; rank 16, 46 : 47; 4096 of 256, rank 16, 56 : 85; 8192 of 512, rank
// 16, 94 : 158; 16384 of 4, rank 16, 108 : 85.) MOE_ADAPTER_FORM overrides the choice for tests
// and tuning.
bool adapter_many(const AdapterArgs& a) {
    if (!adapter_tc_takes(a)) return false;
    if (const char* e = getenv("MOE_ADAPTER_FORM")) {
        if (e[0] == 'm') return true;
        if (e[0] == 'f') return false;
    }
    return static_cast<long long>(a.T) * a.rp >= std::max(65536LL, 1024LL * a.E);
}

template <typename T, typename O>
cudaError_t launch_mma(const AdapterArgs& a, cudaStream_t s) {
    if (adapter_many(a)) return launch_adapter_tc(a, s);
    const bool vec = a.d % 8 == 0 && a.x_stride % 8 == 0 && aligned_to(a.x, 16) && aligned_to(a.a, 16) && a.N % 8 == 0 && a.r % 4 == 0 &&
                     aligned_to(a.b, 8) && aligned_to(a.out, 16) && a.out_stride * sizeof(O) % 16 == 0 && aligned_to(a.base, 16) &&
                     a.base_stride * sizeof(O) % 16 == 0;
    const bool many = a.T >= 24LL * (a.E + 1);  // tiles of 32 rows are mostly full
    if (many) {
        if (a.rp <= 16) return vec ? fused_k<T, O, 2, 2, 1, true>(a, s) : fused_k<T, O, 2, 2, 1, false>(a, s);
        return vec ? fused_k<T, O, 2, 4, 1, true>(a, s) : fused_k<T, O, 2, 4, 1, false>(a, s);
    }
    if (a.rp <= 16) return vec ? fused_k<T, O, 1, 2, 1, true>(a, s) : fused_k<T, O, 1, 2, 1, false>(a, s);
    if (!vec) return fused_k<T, O, 1, 4, 1, false>(a, s);
    const bool wide = a.r % 8 == 0 && aligned_to(a.b, 16);
    if (wide && a.rp % 64 == 0) return fused_k<T, O, 1, 4, 4, true>(a, s);
    if (wide && a.rp % 32 == 0) return fused_k<T, O, 1, 4, 2, true>(a, s);
    return fused_k<T, O, 1, 4, 1, true>(a, s);
}

// Slices of d of the FP32 kernels: warps for all SMs from the tiles there may be, 256 of d at least.
int adapter_slices(int T, int d, int r, int E) {
    const long long units = std::min<long long>(T, (T + F32_ROWS - 1) / F32_ROWS + E + 1) * ((r + F32_RANKS - 1) / F32_RANKS);
    return static_cast<int>(std::max<long long>(1, std::min<long long>({16LL * num_sms() / units, d / 256, 16})));
}

// Rows of v in all slices, at most: no more for fewer rows, so that a workspace serves them too.
// (A unit takes 4 rows or less, so T slices <= 64 SMs where there is more than one slice.)
long long f32_rows(int T) { return std::max<long long>(T, std::min<long long>(16LL * T, 64LL * num_sms())); }

}  // namespace

size_t adapter_workspace(int T, int r, int dtype) {
    const int rp = dtype == MOE_F32 ? (r + 3) / 4 * 4 : (r + 15) / 16 * 16;
    if (dtype == MOE_F32) return 256 + static_cast<size_t>(f32_rows(T)) * rp * 4;
    return 256 + adapter_tc_workspace(T, rp);  // whichever form the call takes
}

cudaError_t launch_adapter(const AdapterArgs& args, cudaStream_t s) {
    AdapterArgs a = args;
    const bool wide = a.out_dtype == MOE_F32;
    if (a.dtype == MOE_F32) {
        a.rp = (a.r + 3) / 4 * 4;
        a.slices = adapter_slices(a.T, a.d, a.r, a.E);
        return launch_f32(a, s);
    }
    a.rp = (a.r + 15) / 16 * 16;
    if (a.dtype == MOE_BF16) return wide ? launch_mma<__nv_bfloat16, float>(a, s) : launch_mma<__nv_bfloat16, __nv_bfloat16>(a, s);
    return wide ? launch_mma<__half, float>(a, s) : launch_mma<__half, __half>(a, s);
}

}  // namespace moe
