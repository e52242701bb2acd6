// 8-bit expert products on the 5th-generation tensor cores (many rows per
// expert). y[i, n] = sa[i] sb[e, n] sum_k a[i, k] b[e, n, k], the sum exact.
//
// sm_103a's tcgen05 has no integer kind, but 8-bit integers are exact in FP16,
// their products (below 2^14) and sums of 1024 of them exact in the FP32
// accumulator. More than that: every partial sum of a row is at most 128 times
// the row's sum of |a|, so a call whose largest row sum is at most 2^17 (rows
// quantised by their maximum stay below it up to a few thousand values) runs
// its whole reduction in one accumulator. Any other call runs in chunks of at
// most 1024, and each chunk's accumulator is added to 32-bit integers in
// registers. Either way the sum is the integer product's, at the FP16 rate.
//
// Roles: output channels are the MMA's M rows, tokens its N columns, one CTA
// pair (cta_group::2) per tile of 256 channels x 256 tokens (or 32, see Form). The tokens are
// widened to FP16 (and gathered) once, by a pass before; the weights stay 8
// bits in HBM, L2 and shared memory, and four warps widen them on their way
// into tensor memory, from where the MMA takes its A operand: weights widened
// into shared memory would add their write and the MMA's read to a shared
// memory that the copies and the tokens already keep half busy.
//
// Warps: 0 copies tokens, 2 weights (TMA), 1 issues MMAs (even CTA), 4-7 (and
// 12-15 with few tokens) widen weights, 8-15 (8-11) hold the integer sums and
// store. A stage is 128 of the
// reduction: 32 KB of tokens and 64 columns of widened weights in tensor memory, which the MMAs free together, and 16 KB of weights in a ring of its
// own, which the widening frees: weights are in shared memory before their
// columns are, so that only the widening lies between two uses of a column.
//
// Measured (one GB300; 1912 TFLOP/s BF16 and 6.8 TB/s by the libraries' product and
// copy): 16384 x 4096 x 4096 268 us without the tokens' pass (2.05 P operations/s: small
// integers in FP16 draw less power than random BF16); 131072 gathered rows of 64 experts,
// 2048 x 2816 SwiGLU, 790 us (1.9 P), the tensor pipe active 81 %; there the widening (1110
// cycles a stage of 1024 MMA cycles) and the last waves bind. 1024 rows of 256 experts,
// 4096 x 4096: 615 us, 6.8 TB/s of weights. The tokens' pass writes two bytes an
// element, 108 us for the 131072 rows: the rate at which this memory takes writes
// alone (a fill of as many bytes takes 141 us).
//
// Every wait is bounded (common.cuh).
#include <math_constants.h>

#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int BK = 128;              // reduction per stage
constexpr int CHUNK_BLOCKS = 8;      // blocks of BK per exact chunk (1024)
constexpr int L1_ONE_CHUNK = 1 << 17;  // row sum of |a| up to which one accumulator is exact
constexpr int CH = 128;              // channels per CTA (MMA rows)
constexpr int W_BYTES = CH * BK;     // a stage's 8-bit weights
constexpr int THREADS = 512;
constexpr int CONV_WARPS = 4;        // warps that widen one stage
constexpr int MAXE = 256;
constexpr int TMEM_COLS = 512;

// A form: tiles of up to NT tokens (MMA columns of the pair).
//   256: compute-bound; one team of widening warps, two of sums (128 integers a thread).
//   32: bound by the weights' bytes; single CTAs (a pair's MMA takes about 160
//       cycles however few its columns), deep weights' ring, two teams of widening
//       warps in turn (one takes 850 cycles a stage, HBM delivers one in 700),
//       one of sums.
template <int NT>
struct Form {
    static constexpr bool WIDE = NT > 32;  // CTA pairs, each CTA half of the tokens
    static constexpr int CTAS = WIDE ? 2 : 1;
    static constexpr int T_HALF = NT / CTAS * 128;  // 64 of the reduction x this CTA's tokens of FP16
    static constexpr int T_BYTES = 2 * T_HALF;
    static constexpr int STAGES = WIDE ? 4 : 7;    // of tokens and of widened weights (64 columns each)
    static constexpr int WSTAGES = WIDE ? 5 : 10;  // of weights
    static constexpr int A_COL = NT;               // tensor-memory columns: accumulator, then widened weights
    static constexpr int TEAMS = WIDE ? 1 : 2;
    static constexpr int EPI_WARPS = WIDE ? 8 : 4;
    static constexpr int EPI_TOK = WIDE ? NT / 2 : NT;  // tokens of an epilogue warp
    // Registers a thread per warpgroup: copies and MMAs, widening, two of sums
    // (or one and the second widening team, where the launch's split is kept).
    static constexpr int REGS_COPY = 64, REGS_CONV = 80, REGS_EPI = 184;
    static constexpr int REGS_SUM = REGS_COPY + REGS_CONV + 2 * REGS_EPI;
    static constexpr int W_OFF = STAGES * T_BYTES;
    static constexpr int NBARS = 2 * STAGES + 2 * WSTAGES + 3;
    static constexpr int BAR_OFF = W_OFF + WSTAGES * W_BYTES;
    static constexpr int MISC_OFF = BAR_OFF + 8 * NBARS;
    static constexpr int TAB_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
    static constexpr int SMEM_BYTES = TAB_OFF + (2 * (MAXE + 1) + 2 * (THREADS / 32)) * 4 + 1024;
    static_assert(A_COL + 64 * STAGES <= TMEM_COLS, "tensor memory");
    static_assert(REGS_SUM <= 4 * 128, "the shares exceed the launch's registers");
    static_assert(T_HALF % 1024 == 0 && SMEM_BYTES <= 232448, "shared memory");
};

struct Int8TcParams {
    CUtensorMap mapW;   // [E, N, K] 8 bits, boxes of 64 channels x 128
    CUtensorMap mapT;   // [M, K] FP16, boxes of a CTA's tokens x 64
    int M, K, N, E, F;  // F: output channels (N, or N / 2 with SwiGLU)
    int nt;             // channel tiles of a pair
    const int32_t* offsets;
    const float* sa;    // [M], gathered
    const float* sb;    // [E, N]
    const int* l1;      // [nl1] largest row sum of |a| per CTA of the tokens' pass
    int nl1;
    void* out;
    int* err;
    unsigned long long timeout_ns;
};

// ---------------------------------------------------------------------------
// tokens: rows gathered and widened to FP16, with their scales
// ---------------------------------------------------------------------------
// Four 8-bit integers as two words of FP16 pairs, exactly: v + 128 in the low
// byte of 1024 + (v + 128), less 1152.
MOE_DEV void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 k = __half2half2(__ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), k);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), k);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

constexpr int TOK_THREADS = 256;

// One warp per row; l1[CTA] receives the largest sum of |a| of its rows. Rows
// from offsets[E] on belong to no expert: their output is zero and nothing
// reads their tokens.
template <typename O>
__global__ void __launch_bounds__(TOK_THREADS)
int8_tokens_kernel(int M, int Ma, int K, int E, int F, const int8_t* __restrict__ a, long long lda,
                   const float* __restrict__ sa, const int32_t* __restrict__ offsets,
                   const int32_t* __restrict__ rows, uint4* __restrict__ tok, float* __restrict__ tsa,
                   O* __restrict__ out, int* __restrict__ l1, int* err) {
    __shared__ unsigned s_l1[TOK_THREADS / 32];
    const int lane = static_cast<int>(lane_id());
    unsigned most = 0;
    pdl_wait();
    pdl_trigger();
    const int step = gridDim.x * (TOK_THREADS / 32);
    int i = blockIdx.x * (TOK_THREADS / 32) + (threadIdx.x >> 5);
    int row = rows != nullptr && i < M ? rows[i] : i;  // of the next turn
    const int covered = offsets != nullptr ? min(max(offsets[E], 0), M) : M;
    for (; i < M; i += step) {
        int src = row;
        row = rows != nullptr && i + step < M ? rows[i + step] : i + step;
        if (i >= covered) {
            for (int n = lane; n < F; n += 32) out[static_cast<long long>(i) * F + n] = from_f32<O>(0.0f);
            continue;
        }
        bool ok = true;
        if (rows != nullptr) {
            ok = src >= 0 && src < Ma;
            if (!ok) {
                if (lane == 0) atomicOr(err, ERRBIT_INDEX);
                src = 0;
            }
        }
        if (lane == 0) tsa[i] = ok ? sa[src] : CUDART_NAN_F;
        const uint2* ar = reinterpret_cast<const uint2*>(a + src * lda);
        uint4* tr = tok + static_cast<long long>(i) * (K / 8);
        unsigned sum = 0;
#pragma unroll 4
        for (int c = lane; c < K / 8; c += 32) {
            const uint2 v = __ldg(ar + c);
            sum = __dp4a(__vabs4(v.x), 0x01010101u, __dp4a(__vabs4(v.y), 0x01010101u, sum));
            uint4 x;
            widen4(v.x, x.x, x.y);
            widen4(v.y, x.z, x.w);
            tr[c] = x;
        }
        most = max(most, __reduce_add_sync(0xffffffffu, sum));
    }
    if (lane == 0) s_l1[threadIdx.x >> 5] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < TOK_THREADS / 32; ++i) most = max(most, s_l1[i]);
        l1[blockIdx.x] = static_cast<int>(most);
    }
}

// ---------------------------------------------------------------------------
// tcgen05 pieces of this kernel
// ---------------------------------------------------------------------------
// Tensor-memory store, 32 lanes x 32 columns of 32 bits: thread i writes lane
// base + i.
MOE_DEV void tc_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
MOE_DEV void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// tc_ld_32x32b_x16 into 16 registers of a larger array.
MOE_DEV void tc_ld_16(uint32_t taddr, uint32_t* r) { tc_ld_32x32b_x16(taddr, *reinterpret_cast<uint32_t(*)[16]>(r)); }

// The issuing warp stays whole: every lane runs its loop, so that descriptors
// and addresses are warp-uniform, and only the tensor instructions are the
// elected lane's. (A loop of one lane took 140 cycles an MMA, whatever its
// size, moving the operands to uniform registers.)
MOE_DEV uint32_t elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(e));
    return e;
}

// Whether the phase of `bar` with parity `parity` is complete, without waiting.
template <bool CLUSTER>
MOE_DEV bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (CLUSTER)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    return ok != 0;
}
// bounded_wait by every lane of a warp, with one outcome.
MOE_DEV bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& w, bool cluster = false) {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, w, cluster)) != 0;
}

// MMA with A in tensor memory (of a pair: each CTA its own 128 rows), FP16
// operands.
template <bool PAIR>
MOE_DEV void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
            "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
            "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}
// Arrive on `bar` (of a pair: in both CTAs) once this thread's MMAs are done.
template <bool PAIR>
MOE_DEV void tc_commit_to(uint32_t bar) {
    if constexpr (PAIR) tc_commit_pair_mc(bar, 3);
    else tc_commit(bar);
}
// FP32 accumulator, FP16 A and B (K-major), M = 128 per CTA; N is added per tile.
constexpr uint32_t idesc0(int ctas) { return (1u << 4) | (static_cast<uint32_t>(ctas * CH >> 4) << 24); }

template <int N>
MOE_DEV void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
MOE_DEV void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// Arrive on an mbarrier of the other CTA, for what tensor memory holds: the
// tcgen05 wait and fence before it order that, so the arrival carries the
// default (CTA) release. A cluster-scope release waits for every access of the
// warp to be visible there: 1.4 k of 2.2 k cycles a stage.
MOE_DEV void mbar_arrive_peer(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

struct Tile {
    int e, row0, n, f0;  // expert, first product row, rows, first output channel of the pair
};

// s_tp: tiles before each expert; s_off: its first row. Channel tiles are
// innermost: neighbouring pairs share a token tile and an expert's weights.
template <int TILE_CH, int NT>
MOE_DEV Tile tile_of(int u, const Int8TcParams& p, const int* s_tp, const int* s_off) {
    const int mt = u / p.nt;
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tp[mid] <= mt) lo = mid;
        else hi = mid;
    }
    Tile t;
    t.e = lo;
    t.row0 = s_off[lo] + (mt - s_tp[lo]) * NT;
    t.n = min(NT, s_off[lo + 1] - t.row0);
    t.f0 = (u - mt * p.nt) * TILE_CH;
    return t;
}

template <int NT, bool SWIGLU, typename O>
__global__ void __launch_bounds__(THREADS, 1) int8_tc_kernel(const __grid_constant__ Int8TcParams p) {
    using G = Form<NT>;
    constexpr int STAGES = G::STAGES, WSTAGES = G::WSTAGES, T_BYTES = G::T_BYTES, T_HALF = G::T_HALF;
    constexpr int OUT_CH = SWIGLU ? CH / 2 : CH;  // output channels per CTA
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + G::BAR_OFF;
    // ready (even CTA): both CTAs' tokens landed and their weights are widened
    auto ready = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };       // tokens and columns read by the MMAs
    auto wfull = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };   // own weights landed
    auto wempty = [&](int s) { return bar0 + 8u * (2 * STAGES + WSTAGES + s); };  // and widened
    const uint32_t acc_full = bar0 + 8u * (2 * STAGES + 2 * WSTAGES), acc_empty = acc_full + 8u, drain_bar = acc_full + 16u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + G::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + G::MISC_OFF + 4);
    int* s_tp = reinterpret_cast<int*>(smem + G::TAB_OFF);
    int* s_off = s_tp + MAXE + 1;
    int* s_l1 = s_off + MAXE + 1;
    int* s_left = s_l1 + THREADS / 32;  // an epilogue warp's first tile that it did not store

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr bool PAIR = G::CTAS == 2;
    const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
    const int unit0 = static_cast<int>(blockIdx.x) / G::CTAS, ustep = static_cast<int>(gridDim.x) / G::CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(ready(s), 1 + G::CTAS * CONV_WARPS);
            mbar_init(empty(s), 1);
        }
        for (int s = 0; s < WSTAGES; ++s) {
            mbar_init(wfull(s), 1);
            mbar_init(wempty(s), CONV_WARPS);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, G::CTAS * G::EPI_WARPS);
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_map(&p.mapW);
        tma_prefetch_map(&p.mapT);
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
            tmem_relinquish();
        }
    }
    pdl_wait();  // the tokens and their scales
    pdl_trigger();
    int l1 = 0;
    for (int i = threadIdx.x; i < p.nl1; i += THREADS) l1 = max(l1, p.l1[i]);
    l1 = __reduce_max_sync(0xffffffffu, l1);
    if (lane == 0) s_l1[warp] = l1;
    if (warp == 2) {  // tiles before each expert, from the clamped offsets
        int before = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int lo = 0, hi = 0;
            if (e < p.E) {
                lo = p.offsets != nullptr ? min(max(p.offsets[e], 0), p.M) : 0;
                hi = p.offsets != nullptr ? min(max(p.offsets[e + 1], 0), p.M) : p.M;
                if (hi < lo) hi = lo;
            }
            const int c = (hi - lo + NT - 1) / NT;
            int x = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (e < p.E) {
                s_tp[e] = before + x - c;
                s_off[e] = lo;
                if (e == p.E - 1) s_off[p.E] = hi;
            }
            before += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) s_tp[p.E] = before;
    }
    __syncwarp();
    tc_fence_before();
    if (PAIR) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = s_tp[p.E] * p.nt;
    const WaitCtx wc{p.err, abort_flag, p.timeout_ns};
    const int kblocks = (p.K + BK - 1) / BK;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) l1 = max(l1, s_l1[i]);
    // blocks per chunk: all, or at most 8 and evenly
    const int nchunks0 = l1 <= L1_ONE_CHUNK ? 1 : (kblocks + CHUNK_BLOCKS - 1) / CHUNK_BLOCKS;
    const int cblocks = (kblocks + nchunks0 - 1) / nchunks0;
    const int nchunks = (kblocks + cblocks - 1) / cblocks;

    if (warp < 4) {
        if (G::WIDE) reg_dec<G::REGS_COPY>();
        if (warp == 0 && lane == 0) {
            // ---------------- tokens (both CTAs) ----------------
            int stage = 0;
            uint32_t phase = 0, issued = 0, last_par = 0;
            bool ok = true;
            for (int u = unit0; u < total && ok; u += ustep) {
                const Tile t = tile_of<G::CTAS * OUT_CH, NT>(u, p, s_tp, s_off);
                const int nh = ((t.n + 15) & ~15) / G::CTAS;  // token columns held by each CTA
                const int trow = t.row0 + rank * nh;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!bounded_wait(empty(stage), phase ^ 1u, wc)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sT = sbase + stage * T_BYTES;
                    if (rank == 0) mbar_expect_tx(ready(stage), G::CTAS * T_BYTES);
                    if (PAIR) {
                        const uint32_t tb = map_shared_rank(ready(stage), 0);
                        tma_load_2d_pair(sT, &p.mapT, kb * BK, trow, tb);
                        tma_load_2d_pair(sT + T_HALF, &p.mapT, kb * BK + 64, trow, tb);
                    } else {
                        tma_load_2d(sT, &p.mapT, kb * BK, trow, ready(stage));
                        tma_load_2d(sT + T_HALF, &p.mapT, kb * BK + 64, trow, ready(stage));
                    }
                    issued |= 1u << stage;
                    last_par = (last_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // every copy has landed before the CTA leaves: seen on the even CTA's
            // barrier, or consumed by the MMAs
            for (int s = 0; s < STAGES; ++s)
                if ((issued >> s) & 1u)
                    bounded_drain(rank == 0 ? ready(s) : empty(s), (last_par >> s) & 1u, p.timeout_ns, p.err);
        } else if (warp == 2 && lane == 0) {
            // ---------------- weights (both CTAs, each its own channels) ----------------
            int stage = 0;
            uint32_t phase = 0, issued = 0, last_par = 0;
            bool ok = true;
            for (int u = unit0; u < total && ok; u += ustep) {
                const Tile t = tile_of<G::CTAS * OUT_CH, NT>(u, p, s_tp, s_off);
                // 64 + 64 channels: a SwiGLU tile's gates and ups, else one run
                const int c0 = t.f0 + rank * OUT_CH, c1 = SWIGLU ? c0 + p.F : c0 + 64;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!bounded_wait(wempty(stage), phase ^ 1u, wc)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sW = sbase + G::W_OFF + stage * W_BYTES;
                    mbar_expect_tx(wfull(stage), W_BYTES);
                    tma_load_3d(sW, &p.mapW, kb * BK, c0, t.e, wfull(stage));
                    tma_load_3d(sW + W_BYTES / 2, &p.mapW, kb * BK, c1, t.e, wfull(stage));
                    issued |= 1u << stage;
                    last_par = (last_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == WSTAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            for (int s = 0; s < WSTAGES; ++s)
                if ((issued >> s) & 1u) bounded_drain(wfull(s), (last_par >> s) & 1u, p.timeout_ns, p.err);
        } else if (warp == 1 && rank == 0) {
            // ---------------- MMA issuer (one warp; even CTA of a pair) ----------------
            const uint32_t elected = elect_one();
            // warp reductions put what came from memory into uniform registers
            const uint32_t d_tmem = __reduce_max_sync(0xffffffffu, tmem);
            const int units = __reduce_max_sync(0xffffffffu, total);
            const int nch = __reduce_max_sync(0xffffffffu, nchunks), cbl = __reduce_max_sync(0xffffffffu, cblocks);
            int stage = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            bool peek = false;  // the stage was seen ready while the one before it was issued
            const uint64_t bdesc0 = smem_desc_sw128(sbase, 16, 1024);
            for (int u = unit0; u < units && ok; u += ustep) {
                const int n = __reduce_max_sync(0xffffffffu, (tile_of<G::CTAS * OUT_CH, NT>(u, p, s_tp, s_off)).n);
                const uint32_t idesc = idesc0(G::CTAS) | (static_cast<uint32_t>(((n + 15) & ~15) >> 3) << 17);
                for (int c = 0; c < nch && ok; ++c) {
                    if (!warp_wait(acc_empty, acc_phase ^ 1u, wc, PAIR)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int kb1 = min((c + 1) * cbl, kblocks);
                    for (int kb = c * cbl; kb < kb1; ++kb) {
                        if (!__all_sync(0xffffffffu, peek) && !warp_wait(ready(stage), phase, wc, PAIR)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const int next = stage + 1 == STAGES ? 0 : stage + 1;
                        const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
                        peek = mbar_test<PAIR>(ready(next), next_phase);
                        const uint64_t bs = bdesc0 + (static_cast<uint64_t>(stage * T_BYTES) >> 4);
                        const uint32_t at = d_tmem + G::A_COL + static_cast<uint32_t>(stage * 64);
                        const uint32_t first = kb == c * cbl ? 0u : 1u;
                        const int steps = min(BK, p.K - kb * BK) / 16;
                        if (elected) {
#pragma unroll
                            for (int ks = 0; ks < BK / 16; ++ks)
                                if (ks < steps)
                                    tc_mma_f16_ta<PAIR>(d_tmem, at + ks * 8, bs + ((ks >> 2) * T_HALF + (ks & 3) * 32) / 16,
                                                        idesc, ks ? 1u : first);
                            tc_commit_to<PAIR>(empty(stage));
                        }
                        __syncwarp();
                        stage = next;
                        phase = next_phase;
                    }
                    if (!ok) break;
                    if (elected) tc_commit_to<PAIR>(acc_full);
                    __syncwarp();
                    acc_phase ^= 1u;
                }
            }
            // the MMAs in flight are done before the CTA leaves
            __syncwarp();
            if (elected) {
                if (PAIR) tc_commit_pair(drain_bar);
                else tc_commit(drain_bar);
                bounded_drain(drain_bar, 0, p.timeout_ns, p.err);
            }
        }
    } else if (warp < 4 + CONV_WARPS || (G::TEAMS == 2 && warp >= 12)) {
        // ---------------- weights: 8 bits in shared memory to FP16 in tensor memory ----------------
        if (G::WIDE) reg_dec<G::REGS_CONV>();
        const int team = warp >= 12 ? 1 : 0;
        const int q = warp & 3;
        // This thread's tensor-memory lane takes one channel of the stage. SwiGLU: a
        // quarter's lanes 0-15 are gates, 16-31 the ups of the same channels.
        const int row = SWIGLU ? (lane < 16 ? 16 * q + lane : 64 + 16 * q + lane - 16) : 32 * q + lane;
        // teams take the stages in turn, across tiles
        int stage = team, ws = team, turn = 0;
        uint32_t phase = 0, wphase = 0;
        bool ok = true;
        for (int u = unit0; u < total && ok; u += ustep) {
            for (int kb = 0; kb < kblocks; ++kb) {
                if (G::TEAMS == 2 && (turn++ & 1) != team) continue;
                // the weights are there ...
                if (!warp_wait(wfull(ws), wphase, wc)) {
                    ok = false;
                    break;
                }
                bool free = mbar_test<false>(empty(stage), phase ^ 1u);
                const uint8_t* wr = smem + G::W_OFF + ws * W_BYTES + row * BK;
                const uint32_t at = tmem + G::A_COL + static_cast<uint32_t>(stage * 64) + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        // 128-byte swizzle: 16-byte chunk j of row r at j ^ (r & 7)
                        const uint4 v = *reinterpret_cast<const uint4*>(wr + (((4 * h + c) ^ (row & 7)) << 4));
                        widen4(v.x, r[8 * c], r[8 * c + 1]);
                        widen4(v.y, r[8 * c + 2], r[8 * c + 3]);
                        widen4(v.z, r[8 * c + 4], r[8 * c + 5]);
                        widen4(v.w, r[8 * c + 6], r[8 * c + 7]);
                    }
                    if (h == 0) {  // ... and the MMAs have read the columns' last content
                        if (!__all_sync(0xffffffffu, free)) free = warp_wait(empty(stage), phase ^ 1u, wc);
                        tc_fence_after();
                    }
                    tc_st_32x32b_x32(at + 32 * h, r);
                }
                tc_wait_st();
                if (!free) {
                    ok = false;
                    break;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(wempty(ws));
                    if (rank == 0) mbar_arrive(ready(stage));
                    else mbar_arrive_peer(map_shared_rank(ready(stage), 0));
                }
                ws += G::TEAMS;
                if (ws >= WSTAGES) {
                    ws -= WSTAGES;
                    wphase ^= 1u;
                }
                stage += G::TEAMS;
                if (stage >= STAGES) {
                    stage -= STAGES;
                    phase ^= 1u;
                }
            }
        }
    } else {
        // ---------------- integer sums and stores ----------------
        if (G::WIDE) reg_inc<G::REGS_EPI>();
        constexpr int TOK = G::EPI_TOK;
        const int q = warp & 3;
        const int c0 = TOK * ((warp - 8) >> 2);  // this warp's token columns [c0, c0 + TOK)
        uint32_t phase = 0;
        bool ok = true;
        int u = unit0;
        for (; u < total; u += ustep) {
            const Tile t = tile_of<G::CTAS * OUT_CH, NT>(u, p, s_tp, s_off);
            const uint32_t ta = tmem + static_cast<uint32_t>(c0) + (static_cast<uint32_t>(q * 32) << 16);
            // one chunk: the FP32 accumulator as it is; several: their integer sum
            uint32_t acc[TOK];
            for (int c = 0; c < nchunks; ++c) {
                if (!warp_wait(acc_full, phase, wc)) {
                    ok = false;
                    break;
                }
                phase ^= 1u;
                tc_fence_after();
                if (c == 0) {
#pragma unroll
                    for (int g = 0; g < TOK / 16; ++g)
                        if (c0 + 16 * g < t.n) tc_ld_16(ta + 16 * g, acc + 16 * g);
                    tc_wait_ld();
                } else {
#pragma unroll
                    for (int g = 0; g < TOK / 16; ++g)
                        if (c0 + 16 * g < t.n) {
                            uint32_t r[16];
                            tc_ld_16(ta + 16 * g, r);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) acc[16 * g + i] += __float2int_rn(__uint_as_float(r[i]));
                        }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(acc_empty);
                    else mbar_arrive_peer(map_shared_rank(acc_empty, 0));
                }
                if (c == 0 && nchunks > 1) {
#pragma unroll
                    for (int i = 0; i < TOK; ++i) acc[i] = __float2int_rn(__uint_as_float(acc[i]));
                }
            }
            if (!ok) break;
            if (nchunks > 1) {
#pragma unroll
                for (int i = 0; i < TOK; ++i) acc[i] = __float_as_uint(static_cast<float>(static_cast<int>(acc[i])));
            }
            // this lane's channel, its scale, and the tokens' scales (lane l: tokens 32 j + l)
            const int oc = SWIGLU ? t.f0 + rank * OUT_CH + 16 * q + (lane & 15) : t.f0 + rank * OUT_CH + 32 * q + lane;
            const bool in = oc < p.F;
            const int ch = SWIGLU && lane >= 16 ? oc + p.F : oc;
            const float sb = in ? __ldg(p.sb + static_cast<long long>(t.e) * p.N + ch) : 0.0f;
            // SwiGLU: lane l + 16 holds the up of lane l's gate
            const float sb2 = SWIGLU ? __shfl_xor_sync(0xffffffffu, sb, 16) : 0.0f;
            const float sbg = lane >> 4 ? sb2 : sb, sbu = lane >> 4 ? sb : sb2;
            float sa[TOK / 32];
#pragma unroll
            for (int j = 0; j < TOK / 32; ++j) {
                const int ti = c0 + 32 * j + lane;
                sa[j] = ti < t.n ? p.sa[t.row0 + ti] : 0.0f;
            }
            O* orow = static_cast<O*>(p.out) + static_cast<long long>(t.row0 + c0) * p.F + oc;
            const int upper = lane >> 4;
            // eight tokens at a time, so that their chains overlap
#pragma unroll
            for (int i = 0; i < TOK; i += 8) {
                if (c0 + i >= t.n) break;
                if constexpr (SWIGLU) {
                    // lanes 0-15 hold gates and finish the even tokens, lanes 16-31 ups and the odd
                    float g[4], up[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float a = __uint_as_float(acc[i + 2 * k]), b = __uint_as_float(acc[i + 2 * k + 1]);
                        const float other = __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
                        const float st = __shfl_sync(0xffffffffu, sa[i >> 5], ((i + 2 * k) & 31) + upper);
                        g[k] = (upper ? other : a) * st * sbg;
                        up[k] = (upper ? b : other) * st * sbu;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int ti = i + 2 * k + upper;
                        const O h = from_f32<O>(g[k] * sigmoid_to<O>(g[k]) * up[k]);
                        if (in && c0 + ti < t.n) orow[static_cast<long long>(ti) * p.F] = h;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float st = __shfl_sync(0xffffffffu, sa[i >> 5], (i + k) & 31);
                        const O h = from_f32<O>(__uint_as_float(acc[i + k]) * st * sb);
                        if (in && c0 + i + k < t.n) orow[static_cast<long long>(i + k) * p.F] = h;
                    }
                }
            }
        }
        if (lane == 0) s_left[warp] = u;
    }

    // A wait ran out: tiles that are not stored become NaN, so that it shows also where
    // nobody reads the error word.
    __syncwarp();
    if (*abort_flag && warp >= 8 && warp < 8 + G::EPI_WARPS) {
        const int c0 = G::EPI_TOK * ((warp - 8) >> 2);
        for (int u = s_left[warp]; u < total; u += ustep) {
            const Tile t = tile_of<G::CTAS * OUT_CH, NT>(u, p, s_tp, s_off);
            const int oc = t.f0 + rank * OUT_CH + (SWIGLU ? 16 * (warp & 3) + (lane & 15) : 32 * (warp & 3) + lane);
            if (oc >= p.F) continue;
            O* orow = static_cast<O*>(p.out) + static_cast<long long>(t.row0 + c0) * p.F + oc;
            for (int i = SWIGLU ? lane >> 4 : 0; i < min(G::EPI_TOK, t.n - c0); i += SWIGLU ? 2 : 1)
                orow[static_cast<long long>(i) * p.F] = from_f32<O>(CUDART_NAN_F);
        }
    }

    // no CTA of the pair leaves while the other may still touch its shared
    // memory, barriers or tensor memory
    __syncwarp();
    tc_fence_before();
    if (PAIR) cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem, TMEM_COLS);
        else tmem_dealloc(tmem, TMEM_COLS);
    }
}

constexpr size_t L1_BYTES = 8192;  // a word per CTA of the tokens' pass
size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

template <int NT, bool SWIGLU, typename O>
int cta_slots(int dev) {  // CTAs, or pairs, that are resident at once
    using G = Form<NT>;
    static int cache[64] = {};
    if (dev < 0 || dev >= 64) return 0;
    if (cache[dev] == 0) {
        int n = -1;
        // the warpgroups' register shares are drawn on what the block is launched with
        cudaFuncAttributes fa{};
        if (cudaFuncGetAttributes(&fa, int8_tc_kernel<NT, SWIGLU, O>) == cudaSuccess &&
            (!G::WIDE || fa.numRegs * 4 >= G::REGS_SUM) &&
            cudaFuncSetAttribute(int8_tc_kernel<NT, SWIGLU, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM_BYTES) ==
                cudaSuccess) {
            if (G::CTAS == 1) return cache[dev] = num_sms();  // a CTA's shared memory fills an SM
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2 * static_cast<unsigned>(num_sms()));
            cfg.blockDim = dim3(THREADS);
            cfg.dynamicSmemBytes = G::SMEM_BYTES;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int c = 0;
            if (cudaOccupancyMaxActiveClusters(&c, int8_tc_kernel<NT, SWIGLU, O>, &cfg) == cudaSuccess && c > 0)
                n = c;
            else
                cudaGetLastError();
        }
        cache[dev] = n;
    }
    return cache[dev] > 0 ? cache[dev] : 0;
}

template <int NT, bool SWIGLU, typename O>
cudaError_t launch_t(const Int8Args& a, cudaStream_t s) {
    int dev = 0;
    cudaGetDevice(&dev);
    const int slots = cta_slots<NT, SWIGLU, O>(dev);
    if (slots <= 0) return cudaErrorInvalidConfiguration;
    uint8_t* ws = reinterpret_cast<uint8_t*>(a.err);
    float* tsa = reinterpret_cast<float*>(ws + 256);
    int* l1 = reinterpret_cast<int*>(ws + 256 + pad256(static_cast<size_t>(a.M) * 4));
    uint8_t* tok = reinterpret_cast<uint8_t*>(l1) + L1_BYTES;
    Int8TcParams p{};
    p.M = a.M; p.K = a.K; p.N = a.N; p.E = a.E;
    p.F = SWIGLU ? a.N / 2 : a.N;
    constexpr int CTAS = Form<NT>::CTAS;
    const int per = CTAS * (SWIGLU ? CH / 2 : CH);
    p.nt = (p.F + per - 1) / per;
    const uint64_t wd[3] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.E)};
    const uint64_t wst[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.K) * a.N};
    const uint32_t wb[3] = {BK, 64, 1};
    const uint64_t td[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.M)};
    const uint64_t tst[1] = {static_cast<uint64_t>(a.K) * 2};
    const uint32_t tb[2] = {64, NT / CTAS};
    if (!encode_tmap_typed(&p.mapW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.b, 3, wd, wst, wb) ||
        !encode_tmap_typed(&p.mapT, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, tok, 2, td, tst, tb))
        return cudaErrorInvalidValue;
    p.offsets = a.offsets;
    const int warps = TOK_THREADS / 32, cap = num_sms() * 8, want = (a.M + warps - 1) / warps;
    const int tgrid = min(min(want, cap), static_cast<int>(L1_BYTES / 4));
    p.sa = tsa; p.sb = a.sb; p.out = a.out;
    p.l1 = l1; p.nl1 = tgrid;
    p.err = a.err;
    p.timeout_ns = wait_timeout_ns();
    cudaError_t e = launch_pdl(int8_tokens_kernel<O>, dim3(tgrid), dim3(TOK_THREADS), 0, s, a.M, a.Ma,
                               a.K, a.E, p.F, a.a, a.lda, a.sa, a.offsets, a.rows, reinterpret_cast<uint4*>(tok), tsa,
                               static_cast<O*>(a.out), l1, a.err);
    if (e != cudaSuccess) return e;
    // tiles: whole ones, and a part for each expert that has rows
    const long long bound = (static_cast<long long>((a.M + NT - 1) / NT) + (a.E > 1 ? (a.E < a.M ? a.E : a.M) : 0)) * p.nt;
    const int grid = static_cast<int>(bound < slots ? (bound > 0 ? bound : 1) : slots);
    if (CTAS == 1)
        return launch_pdl(int8_tc_kernel<NT, SWIGLU, O>, dim3(grid), dim3(THREADS), Form<NT>::SMEM_BYTES, s, p);
    return launch_pdl_cluster(int8_tc_kernel<NT, SWIGLU, O>, dim3(2 * static_cast<unsigned>(grid)), dim3(THREADS),
                              Form<NT>::SMEM_BYTES, s, 2, p);
}

}  // namespace

// Workspace: the error word's 256 bytes, the gathered scales, the tokens'
// pass's row sums, the tokens.
size_t int8_tc_workspace(int M, int K) {
    return 256 + pad256(static_cast<size_t>(M) * 4) + L1_BYTES + static_cast<size_t>(M) * static_cast<size_t>(K) * 2;
}

template <int NT>
static cudaError_t launch_form(const Int8Args& a, cudaStream_t s) {
    switch (a.out_dtype) {
        case MOE_BF16: return a.swiglu ? launch_t<NT, true, __nv_bfloat16>(a, s) : launch_t<NT, false, __nv_bfloat16>(a, s);
        case MOE_F16: return a.swiglu ? launch_t<NT, true, __half>(a, s) : launch_t<NT, false, __half>(a, s);
        default: return a.swiglu ? launch_t<NT, true, float>(a, s) : launch_t<NT, false, float>(a, s);
    }
}

cudaError_t launch_int8_tc(const Int8Args& a, bool wide, cudaStream_t s) {
    return wide ? launch_form<256>(a, s) : launch_form<32>(a, s);
}

}  // namespace moe
