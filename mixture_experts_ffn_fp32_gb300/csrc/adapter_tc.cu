// Low-rank adapters (adapter.cu) of many rows on the 5th-generation tensor cores, 16-bit
// types. Tiles of 128 positions of one adapter.
//
// The first launch computes v = s x A^T and leaves it in pieces of T: a stage is 64 of d, 128
// rows of x (gathered) and the adapter's rank rows of A, copied asynchronously into
// 128-byte-swizzled rows; one thread issues the MMAs (128 x rp x 16), the accumulator [128, rp]
// stays in tensor memory.
//
// The second computes out = base + v B^T in blocks of 128 columns: v's pieces are the A
// operand, [v_1 | v_2 | ..] against the same rows of B, so that the product keeps 16 bits
// of v (FP32 output: 24). Two accumulators take turns: the MMAs of a block run under the
// last one's output. B's rows stand in an order in which a lane that reads 16 x 256 bits of
// tensor memory ends with 8 consecutive columns of its rows.
//
// Measured (one GB300, calls among others): 16384 rows of 16 adapters (a tenth of them without),
// 2048 x 2816, rank 16, 60 us: 20 for v (x at 3 TB/s: a wave of 16 steps a CTA, 4 us before the
// first and 4 for the cluster behind the last) and 39 for the second product, which a plain copy of
// base to out takes 36 for. 8192 rows of 4, 4096 x 4096, rank 64, 61 us (24 + 37). What its loads
// in flight find of L1 counts: see STAGES. Ranks that are no multiple of 8 do not come here: rank 12 68 us, rank 4
// 66, and 60 each when the caller pads them.
//
// Waits for MMAs are bounded (common.cuh). One that runs out ends the CTA's copies into the stages and
// its MMAs, leaves NaN in what is not stored yet, and the MMAs already issued are waited for once more
// (drain) before shared or tensor memory has another use. The other waits always end: cluster
// barriers because every CTA makes the same number of turns, whatever the offsets and whatever
// ran out; allocations of tensor memory because the CTAs of these kernels that an SM has room for
// take its 512 columns at most together, and the kernels here that take more than 256 leave no shared
// memory beside them.
#include <math_constants.h>

#include "adapter.cuh"

namespace moe {
namespace {

constexpr int ROWS = 128, BLOCK = 16384;  // a block: 128 rows of 64 elements of 16 bits

// 16-byte piece c of row r of a 128-byte-swizzled tile.
MOE_DEV uint32_t swizzled(int r, int c) { return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4)); }

// The same of a tile whose rows are 32 bytes (16 elements, one MMA's reduction), 32-byte
// swizzled: no space is lost to ranks below 64.
constexpr int STEP_BYTES = ROWS * 32;
MOE_DEV uint32_t swizzled32(int r, int c) { return static_cast<uint32_t>(r * 32 + ((c ^ (r >> 2 & 1)) << 4)); }
MOE_DEV uint64_t smem_desc_sw32(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= 1ull << 16;
    d |= static_cast<uint64_t>(256 >> 4) << 32;  // between groups of 8 rows
    d |= 1ull << 46;
    d |= 6ull << 61;
    return d;
}

MOE_DEV uint32_t elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(e));
    return e;
}

// FP32 accumulator; A and B K-major, of T; 128 x N.
template <typename T>
constexpr uint32_t idesc(int N) {
    const uint32_t type = __is_same(T, __half) ? 0u : 1u;
    return (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(ROWS >> 4) << 24);
}

// 16 lanes x 32 columns: register 4 j + i of lane (g, t) holds column 8 j + 2 t + (i & 1) of row
// g + 8 (i >> 1).
MOE_DEV void tc_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Waits for the MMAs that the elected lane of the first warp has issued (every commit of theirs has then
// arrived too). By the whole CTA, behind a sync, once.
MOE_DEV void drain(uint32_t bar, const WaitCtx& wc) {
    if (threadIdx.x < 32) {
        if (elect_one()) {  // the same lane at every call
            tc_commit(bar);
            bounded_drain(bar, 0, wc.timeout_ns, wc.err);
        }
        __syncwarp();
    }
    __syncthreads();
    tc_fence_after();
}

MOE_DEV uint8_t* align_1k(uint8_t* p) {
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~static_cast<uintptr_t>(1023));
}

// A cluster of CTAs a tile, each with a part of d. Their sums meet in distributed shared
// memory, in order; each CTA then writes v of its share of the rows, in pieces of T:
//   vp [T][NP][rp], and for FP16 back [T], the inverse of a row's scale.
// Every CTA makes the same number of turns, whatever the offsets: cluster barriers always pair.
// Three stages: the second launch begins under this one, and the loads that it has in flight want
// what shared memory leaves of L1 (five stages, 28 KB of L1: 16384 x 2048 x 2816, rank 16, 71 us for 58).
constexpr int STAGES = 3;

template <typename T, int NP>
__global__ void __launch_bounds__(THREADS, 2)
adapter_shrink_tc_kernel(const __grid_constant__ AdapterArgs a, int turns, int cols, int sums, unsigned long long timeout_ns) {
    constexpr bool SCALED = __is_same(T, __half);
    extern __shared__ uint8_t smem_raw[];
    __shared__ Groups g;
    __shared__ __align__(8) uint64_t bars[STAGES + 1];  // the stages', drain's
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    uint8_t* smem = align_1k(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rp = a.rp, stage_bytes = BLOCK + rp * 128;
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](uint32_t i) { return smem_u32(&bars[i]); };
    const int C = a.cluster, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int clusters = gridDim.x / C, id = blockIdx.x / C;
    if (tid == 0) {
        for (int i = 0; i <= STAGES; ++i) mbar_init(bar(i), 1);
        abort_flag = 0;
        fence_mbarrier_init();
    }
    pdl_wait();
    if (warp == 1) {  // held by no CTA that waits for another launch
        tmem_alloc(smem_u32(&tmem_slot), cols * sums);
        tmem_relinquish();
    }
    tc_fence_before();
    const int tiles = group_table<ROWS>(a, false, g);
    tc_fence_after();
    // Not before every CTA has its columns: those of the second launch allocate theirs before they
    // wait for this one.
    pdl_trigger();
    const uint32_t tmem = tmem_slot;
    const WaitCtx wc{a.err, &abort_flag, timeout_ns};
    const int steps = (a.d + 63) / 64, mine = (steps + C - 1) / C;
    const int k0 = min(a.d, 64 * mine * rank), k1 = min(a.d, k0 + 64 * mine), n = (k1 - k0 + 63) / 64;
    const T* x = static_cast<const T*>(a.x);
    const int c16 = tid & 7, r0 = tid >> 3;  // this thread's 16-byte piece, its rows r0 + 32 i
    float* part = reinterpret_cast<float*>(smem);  // [ROWS][rp], over the stages
    const int share = ROWS / C;
    float* sum = part + ROWS * rp;                 // [share][rp]
    T* vp = static_cast<T*>(a.vp);
    bool alive = true;
    uint32_t it = 0;  // stages consumed: stage it % STAGES, its (it / STAGES)th use
    for (int turn = 0; turn < turns; ++turn) {
        const int tile = turn * clusters + id;
        const bool there_is = tile < tiles;
        if (there_is) {
            const Tile t = tile_of<ROWS>(tile, a, g);
            const T* xr[ROWS / 32];
#pragma unroll
            for (int i = 0; i < ROWS / 32; ++i) {
                const int p = r0 + 32 * i;
                xr[i] = nullptr;
                if (p < t.n) {
                    const int r = row_of(a, t.pos + p);
                    if (r >= 0) xr[i] = x + r * a.x_stride;
                    else if (c16 == 0 && rank == 0) atomicOr(a.err, ERRBIT_INDEX);
                }
            }
            const T* A = static_cast<const T*>(a.a) + static_cast<long long>(t.e) * a.r * a.d;
            auto load = [&](int kb, uint32_t stage) {
                const int k = k0 + 64 * kb + 8 * c16;
                const uint32_t at = sbase + stage * stage_bytes;
#pragma unroll
                for (int i = 0; i < ROWS / 32; ++i) {
                    const bool there = xr[i] != nullptr && k < k1;
                    cp_async_16z(at + swizzled(r0 + 32 * i, c16), there ? xr[i] + k : x, there);
                }
                for (int r = r0; r < rp; r += 32) {
                    const bool there = r < a.r && k < k1;
                    cp_async_16z(at + BLOCK + swizzled(r, c16), there ? A + static_cast<long long>(r) * a.d + k : A, there);
                }
            };
            const bool begun = alive;  // the CTA's
            for (int s = 0; s < STAGES - 1; ++s) {
                if (s < n && alive) load(s, (it + s) % STAGES);
                cp_async_commit();
            }
            for (int kb = 0; kb < n; ++kb, ++it) {
                cp_async_wait<STAGES - 2>();
                fence_proxy_async_smem();
                alive = __syncthreads_and(alive);
                if (!alive) break;
                const uint32_t stage = it % STAGES;
                if (warp == 0) {
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t at = sbase + stage * stage_bytes;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tc_mma_bf16(tmem + kb % sums * cols, smem_desc_sw128(at + 32 * q, 16, 1024),
                                        smem_desc_sw128(at + BLOCK + 32 * q, 16, 1024), idesc<T>(rp), kb >= sums || q > 0);
                        tc_commit(bar(stage));
                    }
                    __syncwarp();
                }
                if (kb + STAGES - 1 < n) {
                    // the stage before this one, once its MMAs have read it
                    const uint32_t last = it + STAGES - 1;
                    if (kb > 0) alive = bounded_wait(bar(last % STAGES), (it - 1) / STAGES & 1, wc);
                    if (alive) load(kb + STAGES - 1, last % STAGES);
                }
                cp_async_commit();
            }
            if (alive && n > 0) alive = bounded_wait(bar((it - 1) % STAGES), (it - 1) / STAGES & 1, wc);
            tc_fence_after();
            cp_async_wait<0>();
            alive = __syncthreads_and(alive);
            if (begun && !alive) drain(bar(STAGES), wc);
            // the stages are free
            const int row = 32 * (warp & 3) + lane;
            for (int c = 16 * (warp >> 2); c < rp; c += 32) {
                float f[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = alive ? 0.0f : CUDART_NAN_F;
                for (int o = 0; o < min(sums, n); ++o) {
                    uint32_t v[16];
                    tc_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + o * cols + c, v);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) f[i] += __uint_as_float(v[i]);
                }
#pragma unroll
                for (int q = 0; q < 16; q += 4) *reinterpret_cast<float4*>(part + row * rp + c + q) = make_float4(f[q], f[q + 1], f[q + 2], f[q + 3]);
            }
            tc_fence_before();
        }
        if (C > 1) cluster_sync();
        else __syncthreads();
        if (there_is) {
            const Tile t = tile_of<ROWS>(tile, a, g);
            const float s = a.scale != nullptr ? __ldg(a.scale + t.e) : 1.0f;
            for (int i = tid; i < share * rp / 4; i += THREADS) {
                const uint32_t at = smem_u32(part + rank * share * rp + 4 * i);
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (C > 1) {
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
                *reinterpret_cast<float4*>(sum + 4 * i) = v;
            }
        }
        if (C > 1) cluster_arrive();  // the others' parts have been read
        __syncthreads();
        if (there_is) {
            const Tile t = tile_of<ROWS>(tile, a, g);
            for (int i = tid; i < share * rp / 8; i += THREADS) {
                const int r = i / (rp / 8), k = i % (rp / 8) * 8, p = rank * share + r;
                if (p >= t.n) continue;
                float scale = 1.0f;
                if constexpr (SCALED) {
                    float most = 0.0f, back;
                    for (int q = 0; q < rp; q += 4) most = largest_finite(*reinterpret_cast<const float4*>(sum + r * rp + q), most);
                    row_scale(most, scale, back);
                    if (k == 0) a.back[t.pos + p] = back;
                }
                T q[8][NP];
#pragma unroll
                for (int h = 0; h < 8; ++h) split<T, NP>(sum[r * rp + k + h] * scale, q[h]);
#pragma unroll
                for (int o = 0; o < NP; ++o)
                    *reinterpret_cast<uint4*>(vp + (static_cast<long long>(t.pos + p) * NP + o) * rp + k) =
                        make_uint4(pack2(q[0][o], q[1][o]), pack2(q[2][o], q[3][o]), pack2(q[4][o], q[5][o]), pack2(q[6][o], q[7][o]));
            }
        }
        if (C > 1) cluster_wait();
        alive = __syncthreads_and(alive);  // the accumulator and the stages are free
        tc_fence_after();
    }
    if (warp == 1) tmem_dealloc(tmem, cols * sums);
}

constexpr int COLS = 128;     // columns of a block
constexpr int B_STAGES = 3;

template <typename T, typename O>
__global__ void __launch_bounds__(THREADS, 2)
adapter_expand_tc_kernel(const __grid_constant__ AdapterArgs a, unsigned long long timeout_ns) {
    constexpr int NP = sizeof(O) == 4 ? 3 : 2;
    constexpr bool SCALED = __is_same(T, __half);
    constexpr int AHEAD = sizeof(O) == 2 ? 2 : 1;  // quarters of a block whose base is under way
    extern __shared__ uint8_t smem_raw[];
    __shared__ Groups g;
    __shared__ __align__(8) uint64_t bars[3];  // the accumulators', drain's
    __shared__ int srow[ROWS];
    __shared__ float sback[SCALED ? ROWS : 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    uint8_t* smem = align_1k(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gi = lane >> 2, ti = lane & 3;
    const int KS = a.rp / 16, a_bytes = NP * KS * STEP_BYTES, b_bytes = KS * STEP_BYTES;
    const uint32_t sA = smem_u32(smem), sB = sA + a_bytes;
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&bars[i]), 1);
        abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), 2 * COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    // what the call was given is complete before the launch before this one could begin
    const int tiles = group_table<ROWS>(a, !a.in_place, g);
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const WaitCtx wc{a.err, &abort_flag, timeout_ns};
    // the tiles' blocks of columns in ranges of equal length over the CTAs, across the tiles' ends:
    // every SM has the same work, whatever the number of tiles
    const int per = (a.N + COLS - 1) / COLS;
    const long long total = static_cast<long long>(tiles) * per;
    const T* vp = static_cast<const T*>(a.vp);
    const O* base = static_cast<const O*>(a.base);
    O* out = static_cast<O*>(a.out);
    const int pieces = a.rp / 8;  // of 16 bytes in a row of B
    bool alive = true;
    uint32_t uses[2] = {0, 0};
    const long long end = total * (blockIdx.x + 1) / gridDim.x;
    for (long long from = total * blockIdx.x / gridDim.x; from < end;) {
        const int tile = static_cast<int>(from / per), c0 = static_cast<int>(from % per) * COLS;
        const int n = static_cast<int>(min(static_cast<long long>(per - c0 / COLS), end - from)), c1 = min(a.N, c0 + COLS * n);
        from += n;
        const Tile t = tile_of<ROWS>(tile, a, g);
        const bool adapted = t.e < a.E;
        const T* B = static_cast<const T*>(a.b) + static_cast<long long>(t.e) * a.N * a.r;
        auto load_b = [&](int b) {
            const uint32_t at = sB + b % B_STAGES * b_bytes;
            for (int i = tid; i < COLS * pieces; i += THREADS) {
                const int col = i / pieces, c = i % pieces, m = col & 31;
                // column 8 i + 2 j + c of 32 at row 8 j + 2 i + c
                const int row = (col & ~31) | (m >> 1 & 3) << 3 | (m >> 3) << 1 | (m & 1);
                const bool there = c0 + COLS * b + col < c1 && 8 * c < a.r;
                cp_async_16z(at + (c >> 1) * STEP_BYTES + swizzled32(row, c & 1), there ? B + static_cast<long long>(c0 + COLS * b + col) * a.r + 8 * c : B, there);
            }
        };
        __syncthreads();  // the last tile's rows have been read
        if (tid < ROWS) {
            srow[tid] = tid < t.n ? row_of(a, t.pos + tid) : -1;
            if (!adapted && c0 == 0 && tid < t.n && srow[tid] < 0) atomicOr(a.err, ERRBIT_INDEX);  // the others': the first launch
        }
        // what a thread that has waited for all MMAs so far copies, none of them reads
        if (adapted && alive) load_b(0);
        pdl_wait();  // v
        pdl_trigger();
        if (adapted && alive) {  // its pieces, in the first block's group
            const int row16 = NP * a.rp / 8;
            for (int i = tid; i < ROWS * row16; i += THREADS) {
                const int p = i / row16, c = i % row16;
                cp_async_16z(sA + (c >> 1) * STEP_BYTES + swizzled32(p, c & 1), vp + (p < t.n ? (t.pos + p) * static_cast<long long>(NP * a.rp) + 8 * c : 0), p < t.n);
            }
            if (SCALED && tid < ROWS) sback[tid] = tid < t.n ? a.back[t.pos + tid] : 1.0f;
        }
        for (int b = 0; b < 2; ++b) {
            if (adapted && alive && b > 0 && b < n) load_b(b);
            cp_async_commit();
        }
        __syncthreads();
        // This warp's 32 rows (its tensor-memory lanes) and 64 of a block's columns.
        const int r32 = 32 * (warp & 3), c64 = 64 * (warp >> 2);
        const O* from_row[2][2];
        O* to_row[2][2];  // NULL: no row
        float back[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int p = r32 + 16 * m + 8 * h + gi, row = srow[p];
                from_row[m][h] = base != nullptr && row >= 0 ? base + row * a.base_stride + c0 + c64 + 8 * ti : nullptr;
                to_row[m][h] = row >= 0 ? out + row * a.out_stride + c0 + c64 + 8 * ti : nullptr;
                back[m][h] = SCALED && adapted ? sback[p] : 1.0f;
            }
        const int width = c1 - c0 - c64 - 8 * ti;  // columns from this lane's first one on
        Cols<O> add[AHEAD][2][2];
        auto load_base = [&](int b, int q, int slot) {
            const int at = COLS * b + 32 * q;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) add[slot][m][h].load(from_row[m][h] + at, from_row[m][h] != nullptr && at < width);
        };
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) load_base(0, q, q);
        for (int b = 0; b <= n; ++b) {
            if (adapted && b < n) {
                cp_async_wait<1>();
                fence_proxy_async_smem();
                alive = __syncthreads_and(alive);
                if (warp == 0 && alive) {
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t d = tmem + (b & 1) * COLS, sb = sB + b % B_STAGES * b_bytes;
                        for (int o = NP - 1; o >= 0; --o)  // the small pieces first: what an addition drops grows with the sum
                            for (int ks = 0; ks < KS; ++ks)
                                tc_mma_bf16(d, smem_desc_sw32(sA + (o * KS + ks) * STEP_BYTES), smem_desc_sw32(sb + ks * STEP_BYTES), idesc<T>(COLS),
                                            o < NP - 1 || ks > 0);
                        tc_commit(smem_u32(&bars[b & 1]));
                    }
                    __syncwarp();
                }
            }
            if (b > 0) {
                const int at = b - 1;
                if (adapted) {
                    if (alive) alive = bounded_wait(smem_u32(&bars[at & 1]), uses[at & 1] & 1, wc);
                    ++uses[at & 1];
                    alive = __all_sync(0xffffffffu, alive);
                    tc_fence_after();
                }
                if (!alive) {
#pragma unroll
                    for (int m = 0; m < 2; ++m) back[m][0] = back[m][1] = CUDART_NAN_F;
                }
                uint32_t again = 0;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int off = COLS * at + 32 * q;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        if (adapted) {
                            uint32_t r[16];
                            tc_ld_16x256b_x4(tmem + (static_cast<uint32_t>(r32 + 16 * m) << 16) + (at & 1) * COLS + c64 + 32 * q, r);
                            tc_wait_ld();
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                F2 acc[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) acc[j] = f2(__uint_as_float(r[4 * j + 2 * h]), __uint_as_float(r[4 * j + 2 * h + 1]));
                                const bool there = to_row[m][h] != nullptr && off < width, nan = any_nan(acc);
                                if (there && !nan) add[q % AHEAD][m][h].add_to(to_row[m][h] + off, acc, back[m][h]);
                                if (there && nan) again |= 1u << (4 * q + 2 * m + h);
                            }
                        } else {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (to_row[m][h] != nullptr && off < width) add[q % AHEAD][m][h].copy_to(to_row[m][h] + off);
                        }
                    }
                    if (AHEAD == 2) load_base(at + 1, q, q);
                    else load_base(q == 0 ? at : at + 1, 1 - q, 0);
                }
                if (again != 0) {
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        if ((again >> i & 1) == 0) continue;
                        const int p = r32 + 8 * (i & 3) + gi, row = srow[p], col = c0 + COLS * at + c64 + 32 * (i >> 2) + 8 * ti;
                        const T* v = vp + (t.pos + p) * static_cast<long long>(NP * a.rp);
                        auto whole = [&](int k) {
                            float s = 0.0f;
#pragma unroll
                            for (int o = 0; o < NP; ++o) s += to_f32(v[o * a.rp + k]);
                            return s;
                        };
                        store_again(out + row * a.out_stride + col, base != nullptr ? base + row * a.base_stride + col : nullptr, whole,
                                    B + static_cast<long long>(col) * a.r, a.r, !alive ? CUDART_NAN_F : SCALED ? sback[p] : 1.0f);
                    }
                }
                tc_fence_before();
            }
            if (adapted && alive && b + 2 < n) load_b(b + 2);  // over the block whose MMAs were waited for
            cp_async_commit();
        }
    }
    pdl_wait();  // never done before the launch before this one
    cp_async_wait<0>();
    if (!__syncthreads_and(alive)) drain(smem_u32(&bars[2]), wc);
    if (warp == 1) tmem_dealloc(tmem, 2 * COLS);
}

long long most_tiles(int T, int E) { return std::min<long long>(T, (T + ROWS - 1) / ROWS + E + 1); }

// Shared memory of the first launch: the stages, and over them the sums [ROWS][rp] and a CTA's share of them.
// A tile of one CTA past rank 96 would keep an SM to itself; halves of it do not.
constexpr int shrink_smem(int rp, int cluster) {
    return std::max(STAGES * (BLOCK + rp * 128), (ROWS + ROWS / cluster) * rp * 4) + 1024;
}
static_assert(ctas_an_sm(shrink_smem(96, 1)) == 2 && ctas_an_sm(shrink_smem(TC_RANKS, 2)) == 2, "two CTAs an SM");

template <typename T, int NP>
cudaError_t shrink(AdapterArgs a, cudaStream_t s) {
    static bool done[64] = {};
    if (!allow_smem(adapter_shrink_tc_kernel<T, NP>, shrink_smem(TC_RANKS, 2), done)) return cudaErrorInvalidValue;
    const long long tiles = most_tiles(a.T, a.E), places = 2LL * num_sms();
    // as many CTAs a tile as there are places for, while each has 256 of d
    a.cluster = 1;
    while (a.cluster < 8 && tiles * a.cluster * 2 <= places && a.d >= 512 * a.cluster) a.cluster *= 2;
    if (a.rp > 96 && a.cluster == 1) a.cluster = 2;
    const int smem = shrink_smem(a.rp, a.cluster);
    const long long clusters = std::min(tiles, places / a.cluster);
    const int turns = static_cast<int>((tiles + clusters - 1) / clusters);
    int cols = 32;
    while (cols < a.rp) cols *= 2;
    const int sums = std::min(4, 256 / cols);  // two CTAs share the 512 columns
    return launch_pdl_cluster(adapter_shrink_tc_kernel<T, NP>, dim3(static_cast<unsigned>(clusters * a.cluster)), dim3(THREADS), smem, s,
                              a.cluster, a, turns, cols, sums, static_cast<unsigned long long>(wait_timeout_ns()));
}

template <typename T, typename O>
cudaError_t launch_t(AdapterArgs a, cudaStream_t s) {
    constexpr int NP = sizeof(O) == 4 ? 3 : 2;
    a.vp = a.v;
    a.back = reinterpret_cast<float*>(static_cast<char*>(a.vp) + static_cast<size_t>(a.T) * NP * a.rp * 2);
    const cudaError_t e = shrink<T, NP>(a, s);
    if (e != cudaSuccess) return e;
    const long long tiles = most_tiles(a.T, a.E), cap = 2LL * num_sms();
    const int smem = (NP + B_STAGES) * (a.rp / 16) * STEP_BYTES + 1024;
    static bool done[64] = {};
    if (!allow_smem(adapter_expand_tc_kernel<T, O>, (NP + B_STAGES) * (TC_RANKS / 16) * STEP_BYTES + 1024, done))
        return cudaErrorInvalidValue;
    return launch_pdl(adapter_expand_tc_kernel<T, O>, dim3(static_cast<unsigned>(std::min(tiles * ((a.N + COLS - 1) / COLS), cap))), dim3(THREADS),
                      smem, s, a, static_cast<unsigned long long>(wait_timeout_ns()));
}

bool on(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

size_t adapter_tc_workspace(int T, int rp) { return static_cast<size_t>(T) * (3 * rp * 2 + 4); }

bool adapter_tc_takes(const AdapterArgs& a) {
    const int eo = a.out_dtype == MOE_F32 ? 4 : 2;
    return a.rp <= TC_RANKS && a.d % 8 == 0 && a.x_stride % 8 == 0 && on(a.x, 16) && on(a.a, 16) && a.r % 8 == 0 &&
           on(a.b, 16) && a.N % 8 == 0 && on(a.out, 16) && a.out_stride * eo % 16 == 0 && on(a.base, 16) && a.base_stride * eo % 16 == 0;
}

cudaError_t launch_adapter_tc(const AdapterArgs& a, cudaStream_t s) {
    const bool wide = a.out_dtype == MOE_F32;
    if (a.dtype == MOE_BF16) return wide ? launch_t<__nv_bfloat16, float>(a, s) : launch_t<__nv_bfloat16, __nv_bfloat16>(a, s);
    return wide ? launch_t<__half, float>(a, s) : launch_t<__half, __half>(a, s);
}

}  // namespace moe
