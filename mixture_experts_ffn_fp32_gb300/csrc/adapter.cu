// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + s_e (x[t] A_e^T) B_e^T,   e the adapter of row t
//
// Rows come grouped by adapter: group e is the positions offsets[e] to offsets[e + 1]
// of `rows`; positions from offsets[E] on have no adapter. Two launches: the first
// computes v = s_e x[t] A_e^T into the workspace (by position, FP32), the second adds
// v B_e^T to base.
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
__global__ void __launch_bounds__(THREADS, 3) adapter_shrink_f32_kernel(const __grid_constant__ AdapterArgs a) {
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

// out = base + v B^T of 64 positions by ranges of 128 columns: a warp has 8 rows, a lane 4
// columns of each. B is turned around on its way into shared memory, 32 ranks at a time.
constexpr int F32_TILE = 64, F32_COLS = 128, F32_STEP = 32;

template <bool VEC>
__global__ void __launch_bounds__(THREADS, 2) adapter_expand_f32_kernel(const __grid_constant__ AdapterArgs a) {
    constexpr int PER = F32_TILE / (THREADS / 32);
    __shared__ Groups g;
    __shared__ __align__(16) float sv[F32_TILE][F32_STEP];
    __shared__ __align__(16) float sb[F32_STEP][F32_COLS + 4];
    __shared__ int srow[F32_TILE];
    const int tiles = group_table<F32_TILE>(a, !a.in_place, g);
    const int lane = static_cast<int>(lane_id()), w = threadIdx.x >> 5;
    const int nb = a.col_parts, len = ((a.N + nb - 1) / nb + F32_COLS - 1) / F32_COLS * F32_COLS;
    const float* base = static_cast<const float*>(a.base);
    float* out = static_cast<float*>(a.out);
    auto column = [&](int i) { return VEC ? 4 * lane + i : lane + 32 * i; };  // of a range, the lane's i-th
    pdl_wait();
    pdl_trigger();
    for (long long u = blockIdx.x; u < static_cast<long long>(tiles) * nb; u += gridDim.x) {
        const Tile t = tile_of<F32_TILE>(static_cast<int>(u / nb), a, g);
        const int c0 = static_cast<int>(u % nb) * len, c1 = min(a.N, c0 + len);
        const int ranks = t.e < a.E ? a.r : 0;
        const float* B = static_cast<const float*>(a.b) + static_cast<long long>(t.e) * a.N * a.r;
        __syncthreads();
        if (threadIdx.x < F32_TILE) srow[threadIdx.x] = threadIdx.x < t.n ? row_of(a, t.pos + threadIdx.x) : -1;
        __syncthreads();
        int row[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) row[i] = srow[w * PER + i];
        for (int n0 = c0; n0 < c1; n0 += F32_COLS) {
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
            float acc[PER][4] = {};
            for (int j0 = 0; j0 < ranks; j0 += F32_STEP) {
                const int steps = min(F32_STEP, (a.rp - j0 + 3) / 4 * 4);  // v is there up to rp, a multiple of 4
                __syncthreads();
                for (int i = threadIdx.x; i < F32_TILE * F32_STEP / 4; i += THREADS) {
                    const int r = i / (F32_STEP / 4), j = i % (F32_STEP / 4) * 4;
                    if (j < steps)
                        *reinterpret_cast<float4*>(&sv[r][j]) = r < t.n ? inner4(a, t.pos + r, j0 + j) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                // a column's ranks by neighbouring threads: read in lines, written 4 banks apart at most
                for (int i = threadIdx.x; i < F32_COLS * steps; i += THREADS) {
                    const int n = i / steps, j = i % steps;
                    sb[j][n] = n0 + n < c1 && j0 + j < a.r ? __ldg(B + static_cast<long long>(n0 + n) * a.r + j0 + j) : 0.0f;
                }
                __syncthreads();
                for (int j = 0; j < steps; j += 4) {
                    float b[4][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < 4; i += VEC ? 4 : 1) {
                            if constexpr (VEC) {
                                const float4 v = *reinterpret_cast<const float4*>(&sb[j + q][4 * lane]);
                                b[q][0] = v.x; b[q][1] = v.y; b[q][2] = v.z; b[q][3] = v.w;
                            } else {
                                b[q][i] = sb[j + q][column(i)];
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

// v = s x A^T of 16 MT positions by 8 NT ranks and one slice of d, by a warp; what reads v
// adds the slices in order.
//   a.v [slices][T][rp], rp = r rounded up to 16 and the ranks behind r zero.
template <int MT, int NT>
struct Shrink {
    // chunks of 32 a warp has in flight, as registers allow
    static constexpr int AHEAD = 2 * MT + NT <= 4 ? 4 : 2 * MT + NT <= 6 ? 3 : 2;
};
template <typename T, int MT, int NT, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) adapter_shrink_mma_kernel(const __grid_constant__ AdapterArgs a) {
    constexpr int WARPS = THREADS / 32, U = Shrink<MT, NT>::AHEAD;
    __shared__ Groups g;
    pdl_wait();
    pdl_trigger();
    const int tiles = group_table<16 * MT>(a, false, g);
    const int lane = static_cast<int>(lane_id()), gi = lane >> 2, ti = lane & 3;
    const int rb = (a.rp + 8 * NT - 1) / (8 * NT), parts = rb * a.slices;
    const int len = ((a.d + a.slices - 1) / a.slices + 31) / 32 * 32;
    const T* x = static_cast<const T*>(a.x);
    const long long units = static_cast<long long>(tiles) * parts, step = static_cast<long long>(gridDim.x) * WARPS;
    // units go to every CTA's first warp, then to the second ones: few spread over all SMs
    for (long long u = static_cast<long long>(threadIdx.x >> 5) * gridDim.x + blockIdx.x; u < units; u += step) {
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
        const T* A = static_cast<const T*>(a.a) + (static_cast<long long>(t.e) * a.r + j0 + gi) * a.d;
        float acc[MT][NT][4] = {};
        uint4 fx[U][MT][2], fa[U][NT];
        auto load = [&](int c, int k) {
            const int at = k + 8 * ti, n = k1 - at;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) fx[c][m][h] = load8<T, VEC>(xr[m][h] + at, xr[m][h] != nullptr ? n : 0);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                fa[c][j] = load8<T, VEC>(A + static_cast<long long>(8 * j) * a.d + at, j0 + 8 * j + gi < a.r ? n : 0);
        };
#pragma unroll
        for (int c = 0; c < U; ++c) load(c, k0 + 32 * c);
        for (int k = k0; k < k1; k += 32 * U) {
#pragma unroll
            for (int c = 0; c < U; ++c) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {  // chunks behind the slice are zeros
                        mma16816<T>(acc[m][j], fx[c][m][0].x, fx[c][m][1].x, fx[c][m][0].y, fx[c][m][1].y, fa[c][j].x, fa[c][j].y);
                        mma16816<T>(acc[m][j], fx[c][m][0].z, fx[c][m][1].z, fx[c][m][0].w, fx[c][m][1].w, fa[c][j].z, fa[c][j].w);
                    }
                load(c, k + 32 * (c + U));
            }
        }
        const float s = a.scale != nullptr ? __ldg(a.scale + t.e) : 1.0f;
        float* out = a.v + (static_cast<long long>(slice) * a.T + t.pos) * a.rp;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 16 * m + 8 * h + gi;
                if (i >= t.n) continue;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int rank = j0 + 8 * j + 2 * ti;
                    if (rank < a.rp)
                        *reinterpret_cast<float2*>(out + i * a.rp + rank) =
                            make_float2(rank < a.r ? s * acc[m][j][2 * h] : 0.0f, rank + 1 < a.r ? s * acc[m][j][2 * h + 1] : 0.0f);
                }
            }
    }
}

// out = base + v B^T. A warp takes 16 MT positions by a range of columns, 32 at a time and
// the next 32 of base under way; its pieces of v stay in shared memory, each lane its own,
// so warps wait for nobody. The warps of a CTA take neighbouring tiles and the same columns:
// where those have one adapter, B comes from L1. Column 2 i + c of a warp's instruction j
// stands for column 8 i + 2 j + c, so that a lane ends with 8 consecutive columns of its rows.
//
// KB: steps of 16 ranks whose B is loaded at once, the next ones under way. From two steps on a
// lane's ranks are 8 consecutive ones of 32 (rp a multiple of 16 KB), else 4 of 16.
template <typename T, typename O, int MT, int KB, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) adapter_expand_mma_kernel(const __grid_constant__ AdapterArgs a) {
    constexpr int WARPS = THREADS / 32, NP = sizeof(O) == 4 ? 3 : 2;
    constexpr bool SCALED = __is_same(T, __half);
    constexpr bool AHEAD = KB == 1;  // the next columns' base too: where B takes few registers
    __shared__ Groups g;
    extern __shared__ __align__(16) uint4 frags[];  // [WARPS][rp / 16][NP][MT][32]
    // what the call was given is complete before the launch before this one could begin
    const int tiles = group_table<16 * MT>(a, !a.in_place, g);
    const int lane = static_cast<int>(lane_id()), w = threadIdx.x >> 5, gi = lane >> 2, ti = lane & 3;
    const int KS = a.rp / 16, nb = a.col_parts, len = ((a.N + nb - 1) / nb + 31) / 32 * 32;
    uint4* frag = frags + w * KS * NP * MT * 32 + lane;
    const O* base = static_cast<const O*>(a.base);
    O* out = static_cast<O*>(a.out);
    bool waited = false;
    for (int u = blockIdx.x; u < (tiles + WARPS - 1) / WARPS * nb; u += gridDim.x) {
        const int tile = u / nb * WARPS + w;
        if (tile >= tiles) continue;
        const Tile t = tile_of<16 * MT>(tile, a, g);
        const int c0 = u % nb * len, c1 = min(a.N, c0 + len);
        const bool adapted = t.e < a.E;
        const T* B = static_cast<const T*>(a.b) + static_cast<long long>(t.e) * a.N * a.r;
        int row[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 16 * m + 8 * h + gi;
                row[m][h] = i < t.n ? row_of(a, t.pos + i) : -1;
            }
        Cols<O, VEC> add[MT][2];
        auto load_base = [&](int n0) {
            const int col = n0 + 8 * ti;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    add[m][h].load(base + row[m][h] * a.base_stride + col, base != nullptr && row[m][h] >= 0 ? c1 - col : 0);
        };
        uint2 fb[KB][4];
        auto rank_of = [&](int ks) { return KB == 1 ? 16 * ks + 4 * ti : 32 * (ks >> 1) + 8 * ti + 4 * (ks & 1); };
        auto load_b = [&](int n0, int ks) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + 8 * (gi >> 1) + 2 * j + (gi & 1);
                const T* p = B + static_cast<long long>(n) * a.r;
                if constexpr (KB == 1) {
                    const int k = rank_of(ks);
                    fb[0][j] = load4<T, VEC>(p + k, adapted && n < c1 ? a.r - k : 0);
                } else {
#pragma unroll
                    for (int q = 0; q < KB; q += 2) {
                        const int k = rank_of(ks + q);
                        const uint4 v = load8<T, VEC>(p + k, adapted && n < c1 ? a.r - k : 0);
                        fb[q][j] = make_uint2(v.x, v.y);
                        fb[q + 1][j] = make_uint2(v.z, v.w);
                    }
                }
            }
        };
        load_b(c0, 0);
        if constexpr (AHEAD) load_base(c0);
        if (!waited) {  // v
            pdl_wait();
            pdl_trigger();
            waited = true;
        }
        float back[MT][2];
        if (adapted) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float scale[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    scale[h] = back[m][h] = 1.0f;
                    if constexpr (SCALED) {
                        const int i = 16 * m + 8 * h + gi;
                        float most = 0.0f;
                        for (int k = 4 * ti; i < t.n && k < a.rp; k += 16) most = largest_finite(inner4(a, t.pos + i, k), most);
                        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                        row_scale(most, scale[h], back[m][h]);
                    }
                }
                for (int ks = 0; ks < KS; ++ks) {
                    T q[2][4][NP];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int i = 16 * m + 8 * h + gi;
                        const float4 v = i < t.n ? inner4(a, t.pos + i, rank_of(ks)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        split<T, NP>(v.x * scale[h], q[h][0]);
                        split<T, NP>(v.y * scale[h], q[h][1]);
                        split<T, NP>(v.z * scale[h], q[h][2]);
                        split<T, NP>(v.w * scale[h], q[h][3]);
                    }
#pragma unroll
                    for (int o = 0; o < NP; ++o)
                        frag[((ks * NP + o) * MT + m) * 32] =
                            make_uint4(pack2(q[0][0][o], q[0][1][o]), pack2(q[1][0][o], q[1][1][o]), pack2(q[0][2][o], q[0][3][o]),
                                       pack2(q[1][2][o], q[1][3][o]));
                }
            }
        }
        for (int n0 = c0; n0 < c1; n0 += 32) {
            Cols<O, VEC> here[MT][2];
            if constexpr (AHEAD) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) here[m][h] = add[m][h];
                load_base(n0 + 32);
            } else {
                load_base(n0);
            }
            float acc[MT][4][4] = {};
            for (int ks = 0; ks < KS; ks += KB) {
                uint2 cur[KB][4];
#pragma unroll
                for (int q = 0; q < KB; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) cur[q][j] = fb[q][j];
                if (ks + KB < KS) load_b(n0, ks + KB);
                else load_b(n0 + 32, 0);
                if (!adapted) break;
#pragma unroll
                for (int q = 0; q < KB; ++q)
#pragma unroll
                    for (int o = 0; o < NP; ++o)
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint4 f = frag[(((ks + q) * NP + o) * MT + m) * 32];
#pragma unroll
                            for (int j = 0; j < 4; ++j) mma16816<T>(acc[m][j], f.x, f.y, f.z, f.w, cur[q][j].x, cur[q][j].y);
                        }
            }
            if constexpr (!AHEAD) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) here[m][h] = add[m][h];
            }
            const int col = n0 + 8 * ti;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (row[m][h] < 0 || col >= c1) continue;
                    float f[8];
                    here[m][h].get(f);
                    if (adapted) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = fmaf(acc[m][i >> 1][2 * h + (i & 1)], back[m][h], f[i]);
                    }
                    Cols<O, VEC>::store(out + row[m][h] * a.out_stride + col, c1 - col, f);
                }
        }
    }
    if (!waited) {  // never done before the launch before it
        pdl_wait();
        pdl_trigger();
    }
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

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

cudaError_t launch_f32(AdapterArgs a, cudaStream_t s) {
    const bool in = a.d % 4 == 0 && a.x_stride % 4 == 0 && aligned_to(a.x, 16) && aligned_to(a.a, 16);
    const long long units = most_tiles(a, F32_ROWS) * ((a.rp + F32_RANKS - 1) / F32_RANKS) * a.slices;
    const cudaError_t e = launch_units(in ? adapter_shrink_f32_kernel<true> : adapter_shrink_f32_kernel<false>, units, 3, 0, s, a);
    if (e != cudaSuccess) return e;
    const bool out = a.N % 4 == 0 && aligned_to(a.out, 16) && a.out_stride % 4 == 0 && aligned_to(a.base, 16) && a.base_stride % 4 == 0;
    const long long tiles = most_tiles(a, F32_TILE);
    a.col_parts = static_cast<int>(std::max<long long>(1, std::min<long long>((a.N + F32_COLS - 1) / F32_COLS, 8LL * num_sms() / tiles)));
    return launch_units(out ? adapter_expand_f32_kernel<true> : adapter_expand_f32_kernel<false>, tiles * a.col_parts, 4, 0, s, a);
}

template <typename T, int MT, bool VEC>
cudaError_t shrink_mma(const AdapterArgs& a, cudaStream_t s) {
    const long long units = most_tiles(a, 16 * MT) * a.slices;
    if (a.rp <= 16) return launch_units(adapter_shrink_mma_kernel<T, MT, 2, VEC>, units, 2, 0, s, a);
    return launch_units(adapter_shrink_mma_kernel<T, MT, 4, VEC>, units * ((a.rp + 31) / 32), 2, 0, s, a);
}

constexpr int EXPAND_SMEM = 200 << 10;  // the pieces of v of 256 ranks and one tile a warp

template <typename T, typename O, int MT, int KB, bool VEC>
cudaError_t expand_mma_k(AdapterArgs a, cudaStream_t s) {
    constexpr int WARPS = THREADS / 32, STEP = (sizeof(O) == 4 ? 3 : 2) * MT * 512 * WARPS;  // of 16 ranks
    static bool done[64] = {};
    if (!allow_smem(adapter_expand_mma_kernel<T, O, MT, KB, VEC>, std::min(16 * STEP, EXPAND_SMEM), done)) return cudaErrorInvalidValue;
    const long long groups = (most_tiles(a, 16 * MT) + WARPS - 1) / WARPS;
    // ranges of columns: as many as give every SM its two CTAs, 32 columns at least
    a.col_parts = static_cast<int>(std::max<long long>(1, std::min<long long>((a.N + 31) / 32, 2LL * num_sms() / groups)));
    return launch_units(adapter_expand_mma_kernel<T, O, MT, KB, VEC>, groups * a.col_parts, 2, static_cast<size_t>(a.rp / 16) * STEP, s, a);
}
template <typename T, typename O, int MT, bool VEC>
cudaError_t expand_mma(const AdapterArgs& a, cudaStream_t s) {
    if constexpr (VEC && MT == 1) {
        if (a.r % 8 == 0 && aligned_to(a.b, 16)) {
            if (a.rp % 64 == 0) return expand_mma_k<T, O, 1, 4, true>(a, s);
            if (a.rp % 32 == 0) return expand_mma_k<T, O, 1, 2, true>(a, s);
        }
    }
    return expand_mma_k<T, O, MT, 1, VEC>(a, s);
}

template <typename T, typename O>
cudaError_t launch_mma(const AdapterArgs& a, cudaStream_t s) {
    if (adapter_tc_takes(a)) return launch_adapter_tc(a, s);
    const bool in = a.d % 8 == 0 && a.x_stride % 8 == 0 && aligned_to(a.x, 16) && aligned_to(a.a, 16);
    const bool out = a.N % 8 == 0 && a.r % 4 == 0 && aligned_to(a.b, 8) && aligned_to(a.out, 16) &&
                     a.out_stride * sizeof(O) % 16 == 0 && aligned_to(a.base, 16) && a.base_stride * sizeof(O) % 16 == 0;
    const bool many = a.T >= 24LL * (a.E + 1);
    cudaError_t e;
    if (many) e = in ? shrink_mma<T, 2, true>(a, s) : shrink_mma<T, 2, false>(a, s);
    else e = in ? shrink_mma<T, 1, true>(a, s) : shrink_mma<T, 1, false>(a, s);
    if (e != cudaSuccess) return e;
    // two tiles a warp while their pieces of v leave room for two CTAs an SM
    if (many && a.rp / 16 * (sizeof(O) == 4 ? 3 : 2) * 8192 <= 96 << 10) return out ? expand_mma<T, O, 2, true>(a, s) : expand_mma<T, O, 2, false>(a, s);
    return out ? expand_mma<T, O, 1, true>(a, s) : expand_mma<T, O, 1, false>(a, s);
}

// Slices of d: warps for all SMs from the tiles there may be, 256 of d at least.
int adapter_slices(int T, int d, int r, int E) {
    const long long units = ((T + 31) / 32 + std::min<long long>(E, T)) * ((r + 31) / 32), warps = 16LL * num_sms();
    return static_cast<int>(std::max<long long>(1, std::min<long long>({(warps + units - 1) / units, d / 256, 16})));
}

}  // namespace

size_t adapter_workspace(int T, int d, int r, int E) {
    return 256 + static_cast<size_t>(T) * ((r + 15) / 16 * 16) * 4 * std::max(adapter_slices(T, d, r, E), adapter_tc_slices(T, d, E));
}

cudaError_t launch_adapter(const AdapterArgs& args, cudaStream_t s) {
    AdapterArgs a = args;
    a.rp = (a.r + 15) / 16 * 16;
    a.slices = adapter_slices(a.T, a.d, a.r, a.E);
    if (a.dtype == MOE_F32) return launch_f32(a, s);
    const bool wide = a.out_dtype == MOE_F32;
    if (a.dtype == MOE_BF16) return wide ? launch_mma<__nv_bfloat16, float>(a, s) : launch_mma<__nv_bfloat16, __nv_bfloat16>(a, s);
    return wide ? launch_mma<__half, float>(a, s) : launch_mma<__half, __half>(a, s);
}

}  // namespace moe
