// Group-limited routing from given logits, forward and backward.
//
//   s = sigmoid(r), or softmax of r over the E experts;  c = s + b
//   an expert counts where r > -inf and c > -inf (a NaN never does)
//   group score = sum of the group's n largest c (n = 1 or 2; what it has of them)
//   the topk_groups best groups stay, the K largest c of their experts are taken,
//   equal values rank the lower index first; slots left over hold id -1, weight 0
//   w = scale s_sel, or scale s_sel / sum s_sel
//
// Which experts are taken is decided as 64-bit arithmetic decides it, without
// paying for it: FP32 scores come with an error bound, and only a token whose
// taken ranks, or the groups on either side of the border, lie within it (about
// one in five hundred on random logits) takes FP64 scores, and those only for
// the experts that could be concerned: a warp's FP64 exponential alone is two
// thousand cycles here, and a token all of whose choices took one held up the
// whole batch for 10 us.
//
// One warp per token, E / 32 consecutive experts a lane: scores, the groups'
// two best by shuffles, then the lanes' sorted keys popped by one integer
// maximum over the warp a rank. Bound by instructions (1020 a token of 256 experts,
// 75 of them accesses to registers spilled at the 64 a thread that eight CTAs an SM
// leave; 69 % of the issue slots busy) and, below a few thousand tokens, by the
// latency of that chain. Measured, alone with cold caches: 16384 x 256 sigmoid, 8
// groups, bias 23-28 us, 21 among other calls (3 us of it for the reads at the copy
// rate); 128 tokens 6 us (4 among others); 10007 x 96 softmax of BF16 logits 13.5-16 us;
// groups of 9 experts, which fill no lanes, 7711 x 144, 22 us. The gradient of a raw
// softmax, 16384 x 256: 13-15 us, 11-12 among others (its bytes: 5); of the other forms,
// which read the taken logits alone, 7.7 among others (its bytes: 2.7). It takes 565
// instructions a token in 67 % of the issue slots, and waits for its loads most.
#include <math_constants.h>

#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

// Small CTAs, many of them: the rare token that takes FP64 holds up three others.
constexpr int WARPS = 4;
constexpr unsigned FULL = 0xffffffffu;

// Largest value over the warp (no NaN among them).
MOE_DEV float warp_max(float v) {
    const int u = __float_as_int(v);  // order as signed integers: negative floats reversed
    const int k = __reduce_max_sync(FULL, u ^ ((u >> 31) & 0x7fffffff));
    return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}
template <typename F>
MOE_DEV F warp_add(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
// A NaN becomes -inf: never taken.
MOE_DEV float clean(float r) { return fmaxf(r, -CUDART_INF_F); }

struct Params {
    int T, E, K, G, gs, TG, rank, softmax, renorm;
    // lg = 2^lsh lanes a group: those that hold its experts where groups fill whole
    // lanes (whole), else as many as 32 lanes give G groups
    int lg, lsh, whole;
    int per_group;  // 2^16 / gs, rounded up: expert e < 256 is in group e per_group / 2^16
    float scale;
    long long stride;
    const float* bias;
};

template <int VPL, typename T, bool VEC>
MOE_DEV void load_row(const T* row, int lane, int E, float (&r)[VPL]) {
    const int e0 = lane * VPL;
    if constexpr (VEC) {
        constexpr int B = VPL * sizeof(T) >= 16 ? 16 : VPL * sizeof(T);
        constexpr int N = B / sizeof(T);
        if (e0 < E) {
#pragma unroll
            for (int i = 0; i < VPL; i += N) {
                alignas(16) T v[N];
                if constexpr (B == 16)
                    *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(row + e0 + i);
                else if constexpr (B == 8)
                    *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(row + e0 + i);
                else if constexpr (B == 4)
                    *reinterpret_cast<uint32_t*>(v) = *reinterpret_cast<const uint32_t*>(row + e0 + i);
                else
                    v[0] = row[e0 + i];
#pragma unroll
                for (int j = 0; j < N; ++j) r[i + j] = clean(to_f32(v[j]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) r[i] = -CUDART_INF_F;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) r[i] = e0 + i < E ? clean(to_f32(row[e0 + i])) : -CUDART_INF_F;
    }
}

// The two largest of (a1, a2) and (b1, b2); no NaN among them.
MOE_DEV float least(float a, float b) { return fminf(a, b); }
MOE_DEV float most(float a, float b) { return fmaxf(a, b); }
MOE_DEV long long least(long long a, long long b) { return a < b ? a : b; }
MOE_DEV long long most(long long a, long long b) { return a < b ? b : a; }
template <typename F>
MOE_DEV void merge2(F& a1, F& a2, F b1, F b2) {
    const F lo = least(a1, b1);
    a1 = most(a1, b1);
    a2 = most(most(a2, b2), lo);
}

// 1 / (1 + 2^(-r log2 e)) on the special-function unit; the error bounds in the
// kernel count it. Beyond 87 it is 0 or 1.
MOE_DEV float sigmoid_of(float r) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(r * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
}

// A choice in FP32 from its logit and bias (no NaN), the same wherever it is
// computed.
MOE_DEV float choice(const Params& p, float r, float b, float m, float inv) {
    const float s = p.softmax ? __fmul_rn(r == m ? 1.0f : expf(r - m), inv) : sigmoid_of(r);
    return __fadd_rn(s, r > -CUDART_INF_F ? b : -CUDART_INF_F);
}

// The biases of a lane's experts (0 without a bias, -inf for a NaN and past the last).
template <int VPL, bool VEC>
MOE_DEV void lane_bias(const Params& p, int lane, float (&b)[VPL]) {
    if (p.bias == nullptr) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) b[i] = lane * VPL + i < p.E ? 0.0f : -CUDART_INF_F;
    } else {
        load_row<VPL, float, VEC>(p.bias, lane, p.E, b);
    }
}

// Choices of a row; m, z and inv: softmax maximum, denominator and its
// reciprocal.
template <int VPL>
MOE_DEV void choices(const Params& p, const float (&r)[VPL], const float (&b)[VPL], float (&c)[VPL], float& m, float& z,
                     float& inv) {
    m = 0.0f;
    z = inv = 1.0f;
    if (p.softmax) {
        float mx = r[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) mx = fmaxf(mx, r[i]);
        m = warp_max(mx);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            // equal to the maximum: 1, also where both are infinite
            c[i] = r[i] == m ? 1.0f : expf(r[i] - m);
            s += r[i] == -CUDART_INF_F ? 0.0f : c[i];
        }
        z = warp_add(s);
        if (z == 0.0f) z = 1.0f;
        inv = 1.0f / z;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if (p.softmax) {
            c[i] = __fadd_rn(__fmul_rn(c[i], inv), r[i] > -CUDART_INF_F ? b[i] : -CUDART_INF_F);
        } else {
            c[i] = choice(p, r[i], b[i], m, inv);
        }
    }
}

// Groups that stay, as a mask, from the score of group `lane` (none where the
// group has no expert).
template <typename F>
MOE_DEV unsigned kept_groups(const Params& p, int lane, F mine) {
    int before = 0;  // groups that rank before mine
    for (int g = 0; g < p.G; ++g) {
        const F o = __shfl_sync(FULL, mine, g);
        before += (o > mine || (o == mine && g < lane)) ? 1 : 0;
    }
    return __ballot_sync(FULL, lane < p.G && before < p.TG);
}

// The two best of each group, in F's order: those of the lane's group in
// every lane where groups are whole lanes, else those of group `lane`.
template <typename F, int VPL>
MOE_DEV void group_best(const Params& p, int lane, const F (&c)[VPL], F none, F& a1, F& a2) {
    if (p.whole) {
        a1 = c[0];
        a2 = none;
#pragma unroll
        for (int i = 1; i < VPL; ++i) merge2(a1, a2, c[i], none);
        for (int o = 1; o < p.lg; o <<= 1)
            merge2(a1, a2, __shfl_xor_sync(FULL, a1, o), __shfl_xor_sync(FULL, a2, o));
    } else {
        F m1 = none, m2 = none;
        for (int g = 0; g < p.G; ++g) {
            F b1 = none, b2 = none;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if ((lane * VPL + i) / p.gs == g) merge2(b1, b2, c[i], none);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
                merge2(b1, b2, __shfl_xor_sync(FULL, b1, o), __shfl_xor_sync(FULL, b2, o));
            if (lane == g) {
                m1 = b1;
                m2 = b2;
            }
        }
        a1 = m1;
        a2 = m2;
    }
}

// The two best of a group of any size, in every lane of the group: from a copy
// in shared memory, every lg-th expert a lane. Out of line, as few routings have
// groups that do not fill lanes.
template <int VPL>
__device__ __noinline__ float2 any_group_best(const Params* pp, const float* c, float* copy) {
    const Params& p = *pp;
    const int lane = static_cast<int>(lane_id()), g = lane >> p.lsh;
#pragma unroll
    for (int i = 0; i < VPL; ++i) copy[lane * VPL + i] = c[i];
    __syncwarp();
    float a1 = -CUDART_INF_F, a2 = a1;
    if (g < p.G)
        for (int j = lane & (p.lg - 1); j < p.gs; j += p.lg) merge2(a1, a2, copy[g * p.gs + j], -CUDART_INF_F);
    for (int o = 1; o < p.lg; o <<= 1) merge2(a1, a2, __shfl_xor_sync(FULL, a1, o), __shfl_xor_sync(FULL, a2, o));
    __syncwarp();
    return make_float2(a1, a2);
}

// The groups to keep, as a mask; lo, hi: the lowest kept and the highest
// dropped score (-inf: none); mag: the largest |a| + |b| of a group's two best;
// mine: the score of the lane's group, a2 its second best.
template <int VPL>
MOE_DEV unsigned choose_groups(const Params& p, int lane, const float (&c)[VPL], float* copy, float& lo, float& hi,
                               float& mag, float& mine, float& a2) {
    float a1;
    if (p.whole) {
        group_best<float, VPL>(p, lane, c, -CUDART_INF_F, a1, a2);
    } else {
        float tmp[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) tmp[i] = c[i];
        const float2 best = any_group_best<VPL>(&p, tmp, copy);
        a1 = best.x;
        a2 = best.y;
    }
    mine = (p.rank == 2 && a2 > -CUDART_INF_F) ? a1 + a2 : a1;
    float of = __shfl_sync(FULL, mine, lane << p.lsh & 31);  // of group `lane`
    if (lane >= p.G) of = -CUDART_INF_F;
    const unsigned keep = kept_groups<float>(p, lane, of);
    const bool kept = (keep >> lane) & 1u;
    lo = -warp_max(kept ? -of : -CUDART_INF_F);
    hi = warp_max(lane < p.G && !kept ? of : -CUDART_INF_F);
    mag = warp_max((a1 > -CUDART_INF_F ? fabsf(a1) : 0.0f) + (a2 > -CUDART_INF_F ? fabsf(a2) : 0.0f));
    return keep;
}

// Integers that order as the floats do, and back.
MOE_DEV float key_value(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

MOE_DEV long long order_key(double v) {
    const long long u = __double_as_longlong(v + 0.0);
    return u ^ ((u >> 63) & 0x7fffffffffffffffLL);
}
MOE_DEV double key_value(long long k) { return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffLL)); }
constexpr long long NONE64 = static_cast<long long>(0x8000000000000000ull);

// Scores rise with their logits: without a bias the logits rank (the sum turns
// -0 into 0, which it equals but whose bits lie below).
template <int VPL>
MOE_DEV void logits_rank(const float (&r)[VPL], float (&c)[VPL]) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = c[i] > -CUDART_INF_F ? __fadd_rn(r[i], 0.0f) : -CUDART_INF_F;
}

// How far apart two logits a >= b must be for FP64 to tell their scores apart
// (infinite where it may not: sigmoids near 1, scores below its range).
MOE_DEV float logit_slack(const Params& p, float m, float a, float b) {
    if (p.softmax) return m - b < 690.0f ? 1e-11f : CUDART_INF_F;
    return b > -690.0f && a < 80.0f ? 1e-11f + 4e-16f * __expf(a) : CUDART_INF_F;
}

// Groups ranked by their best logits tie exactly at the border, at `tie`: whether
// FP64 could take a group above or below for equal to them too. `mine`: the score of
// the lane's group.
__device__ __noinline__ bool tied_border_near(const Params* pp, float m, float mine, float tie) {
    const Params& p = *pp;
    const int lane = static_cast<int>(lane_id());
    float of = __shfl_sync(FULL, mine, lane << p.lsh & 31);  // of group `lane`
    if (lane >= p.G) of = -CUDART_INF_F;
    const float up = -warp_max(of > tie ? -of : -CUDART_INF_F), down = warp_max(of < tie ? of : -CUDART_INF_F);
    return (__any_sync(FULL, of > tie) && !(up - tie > logit_slack(p, m, up, tie))) ||
           (down > -CUDART_INF_F && !(tie - down > logit_slack(p, m, tie, down)));
}

// Sorts a lane's keys in descending order (Batcher's odd-even merge).
MOE_DEV void order2(int& a, int& b) {
    const int hi = max(a, b);
    b = min(a, b);
    a = hi;
}
template <int VPL>
MOE_DEV void sort_desc(int (&k)[VPL]) {
    if constexpr (VPL == 2) {
        order2(k[0], k[1]);
    } else if constexpr (VPL == 4 || VPL == 8) {
#pragma unroll
        for (int o = 0; o < VPL; o += 4) {
            order2(k[o], k[o + 1]);
            order2(k[o + 2], k[o + 3]);
            order2(k[o], k[o + 2]);
            order2(k[o + 1], k[o + 3]);
            order2(k[o + 1], k[o + 2]);
        }
        if constexpr (VPL == 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) order2(k[i], k[i + 4]);
            order2(k[2], k[4]);
            order2(k[3], k[5]);
            order2(k[1], k[2]);
            order2(k[3], k[4]);
            order2(k[5], k[6]);
        }
    }
}

// The n largest choices, roughly: keys of the choice's upper 24 bits and, below
// them, 255 less the expert, so that one integer maximum over the warp names
// the expert and only its lane drops its first. Lane k receives the k-th key
// (below FIRST, which -inf and the lanes past n are: none); the caller puts
// what the dropped bits leave open in order.
constexpr int EMPTY = static_cast<int>(0x80000000u), FIRST = static_cast<int>(0x80800000u);
template <int VPL>
MOE_DEV int take_rough(const float (&c)[VPL], int lane, int n) {
    int k[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int u = __float_as_int(c[i]);
        k[i] = ((u ^ ((u >> 31) & 0x7fffffff)) & ~255) | (255 - (lane * VPL + i));
    }
    sort_desc<VPL>(k);
    int key = EMPTY;
    for (int j = 0; j < n; ++j) {
        const int v = __reduce_max_sync(FULL, k[0]);
        if (lane == j) key = v;
        if (k[0] == v) {
#pragma unroll
            for (int i = 0; i + 1 < VPL; ++i) k[i] = k[i + 1];
            k[VPL - 1] = EMPTY;
        }
    }
    return key;
}

// exp(a - b) with the rounding of the difference put back (a - b = d + e).
MOE_DEV float exp_diff(float a, float b) {
    const float d = a - b, bv = a - d, e = (a - (d + bv)) + (bv - b);
    return expf(d) * (1.0f + (isfinite(e) ? e : 0.0f));
}

// Weight over scale of the selected expert of this lane (r; `there` where the
// lane has one), and q = s / sum of the selected s. The sum is taken relative
// to its largest part, so that scores below FP32's range still share it.
MOE_DEV float selected_score(const Params& p, bool there, float r, float m, float z, float& q) {
    const float top = warp_max(there ? r : -CUDART_INF_F);
    float s, part;
    if (p.softmax) {
        s = !there ? 0.0f : r == m ? 1.0f / z : exp_diff(r, m) / z;
        part = !there ? 0.0f : r == top ? 1.0f : exp_diff(r, top);
    } else {
        const float base = fminf(top, 0.0f), ex = expf(-fabsf(r)), den = 1.0f / (1.0f + ex);
        s = !there ? 0.0f : r >= 0.0f ? den : ex * den;
        part = !there ? 0.0f : r >= 0.0f ? den : (base == 0.0f ? ex : expf(r - base)) * den;
    }
    const float sum = warp_add(part);
    q = there ? part / sum : 0.0f;
    return s;
}

// Ids and weights of token t: lane k holds the k-th id and its logit.
MOE_DEV void write_token(const Params& p, long long t, int lane, int id, float rk, float m, float z, int32_t* idx,
                         float* w) {
    const bool there = lane < p.K && id >= 0;
    float q;
    const float s = selected_score(p, there, rk, m, z, q);
    if (lane < p.K) {
        idx[t * p.K + lane] = there ? id : -1;
        w[t * p.K + lane] = there ? p.scale * (p.renorm ? q : s) : 0.0f;
    }
}

// An exact score plus bias: what FP64 makes of a logit (a softmax's without its
// denominator, which is common where there is no bias).
__device__ __noinline__ double exact_choice(int softmax, float r, float m, float b) {
    const double ex = exp(softmax ? static_cast<double>(r) - static_cast<double>(m) : -static_cast<double>(r));
    return (softmax ? (r == m ? 1.0 : ex) : 1.0 / (1.0 + ex)) + static_cast<double>(b);
}

// The groups to keep where some scores lie within `tol` of the border: those
// groups' best experts get FP64 scores. False: there are several candidates for
// a group's best, or a softmax with a bias.
template <typename T>
__device__ __noinline__ bool choose_groups_exact(const Params* pp, const T* row, float m, float inv, float mine, float a2,
                                                 float lo, float hi, float tol, unsigned* keep) {
    const Params& p = *pp;
    if (p.softmax && p.bias != nullptr) return false;
    const int lane = static_cast<int>(lane_id()), g = lane >> p.lsh;
    const bool near = mine > -CUDART_INF_F && mine >= lo - 2.0f * tol && mine <= hi + 2.0f * tol;
    const bool pair = p.rank == 2 && a2 > -CUDART_INF_F;
    const float edge = pair ? a2 : mine;
    int n = 0;
    float ri = 0.0f, bi = 0.0f, rj = 0.0f, bj = 0.0f;
    if (near)  // which lane of the group looks at which expert does not matter
        for (int j = lane & (p.lg - 1); j < p.gs; j += p.lg) {
            const int e = g * p.gs + j;
            const float r = clean(to_f32(row[e])), b = p.bias != nullptr ? clean(p.bias[e]) : 0.0f;
            const float c = choice(p, r, b, m, inv);
            if (c > -CUDART_INF_F && c >= edge - 2.0f * tol) {
                ++n;
                rj = ri;
                bj = bi;
                ri = r;
                bi = b;
            }
        }
    int all = n;
    for (int o = 1; o < p.lg; o <<= 1) all += __shfl_xor_sync(FULL, all, o);
    if (__any_sync(FULL, near && all != (pair ? 2 : 1))) return false;
    double x = n ? exact_choice(p.softmax, ri, m, bi) : 0.0;
    if (__any_sync(FULL, n > 1)) x += n > 1 ? exact_choice(p.softmax, rj, m, bj) : 0.0;  // both in one lane
    for (int o = 1; o < p.lg; o <<= 1) x += __shfl_xor_sync(FULL, x, o);
    // the others lie clear on either side: kept above all, or behind all
    const long long key = near ? order_key(x) : mine > hi ? 0x7fffffffffffffffLL : mine > -CUDART_INF_F ? NONE64 + 1 : NONE64;
    long long of = __shfl_sync(FULL, key, lane << p.lsh & 31);
    if (lane >= p.G) of = NONE64;
    *keep = kept_groups<long long>(p, lane, of);
    return true;
}

// Puts the K + 1 first ranks (lanes 0 to K) in their exact order: some are close,
// but none behind them is. One FP64 score a lane.
__device__ __noinline__ void order_exact(const Params& p, int lane, float m, float b, int& id, float& rk) {
    long long key = NONE64;
    if (lane <= p.K && id >= 0) key = order_key(exact_choice(p.softmax, rk, m, b));
    int rank = 0, src = lane;
    for (int j = 0; j <= p.K; ++j) {
        const long long o = __shfl_sync(FULL, key, j);
        const int oid = __shfl_sync(FULL, id, j);
        rank += (o > key || (o == key && oid < id)) ? 1 : 0;
    }
    if (key == NONE64) rank = lane;
    for (int j = 0; j <= p.K; ++j)
        if (__shfl_sync(FULL, rank, j) == lane) src = j;
    id = __shfl_sync(FULL, id, src);
    rk = __shfl_sync(FULL, rk, src);
}

// A token decided in FP64: the rare token whose FP32 choices lie within their
// error. The choices are 64-bit integers in the doubles' order; those that a
// decision could concern are replaced by exact ones before it is taken. Out of line, so that its registers are not the
// common path's.
template <int VPL, typename T, bool VEC>
__device__ __noinline__ void route_exact(const Params* pp, long long t, const T* row, int32_t* idx, float* w) {
    const Params& p = *pp;
    const int lane = static_cast<int>(lane_id());
    float r[VPL], b[VPL], c[VPL], m, z, inv;
    load_row<VPL, T, VEC>(row, lane, p.E, r);
    lane_bias<VPL, VEC>(p, lane, b);
    choices<VPL>(p, r, b, c, m, z, inv);
    // what two near FP32 choices around v can be apart
    auto slack = [&](float v) { return (p.bias != nullptr ? 0x1p-16f : 0.0f) + 0x1p-13f * fabsf(v) + 1e-35f; };
    // A softmax's denominator is common: without a bias the exponentials decide.
    double z64 = 1.0;
    if (p.softmax && p.bias != nullptr) {
        z64 = 0.0;
#pragma unroll 1
        for (int i = 0; i < VPL; ++i) {
            float ri = r[0];
#pragma unroll
            for (int j = 1; j < VPL; ++j)
                if (j == i) ri = r[j];
            if (ri > -CUDART_INF_F) z64 += ri == m ? 1.0 : exp(static_cast<double>(ri) - static_cast<double>(m));
        }
        z64 = warp_add(z64);
    }
    const double unit = p.softmax && p.bias == nullptr ? static_cast<double>(z) : 1.0;  // FP32 choices to that scale
    long long h[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        h[i] = c[i] > -CUDART_INF_F ? order_key(static_cast<double>(c[i]) * unit) : NONE64;
    unsigned done = 0;
    auto make_exact = [&](unsigned need) {
        need &= ~done;
        done |= need;
        while (__any_sync(FULL, need != 0)) {
            const int at = __ffs(need) - 1;  // -1: nothing left in this lane
            need &= need - 1;
            float ri = r[0], bi = b[0];
#pragma unroll
            for (int j = 1; j < VPL; ++j)
                if (j == at) {
                    ri = r[j];
                    bi = b[j];
                }
            const double x = p.softmax ? static_cast<double>(ri) - static_cast<double>(m) : -static_cast<double>(ri);
            const double ex = p.softmax && ri == m ? 1.0 : exp(x);
            const double s = p.softmax ? (p.bias != nullptr ? ex / z64 : ex) : 1.0 / (1.0 + ex);
            const long long k = order_key(p.bias != nullptr ? s + static_cast<double>(bi) : s);
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (j == at) h[j] = k;
        }
    };
    if (p.G > 1) {
        float f1, f2;
        group_best<float, VPL>(p, lane, c, -CUDART_INF_F, f1, f2);
        unsigned need = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int g = min((lane * VPL + i) / p.gs, 31);
            const float x1 = p.whole ? f1 : __shfl_sync(FULL, f1, g), x2 = p.whole ? f2 : __shfl_sync(FULL, f2, g);
            const float edge = p.rank == 2 && x2 > -CUDART_INF_F ? x2 : x1;
            if (c[i] > -CUDART_INF_F && !(c[i] < edge - slack(edge))) need |= 1u << i;
        }
        make_exact(need);
        long long a1, a2;
        group_best<long long, VPL>(p, lane, h, NONE64, a1, a2);
        long long g = p.rank == 2 && a2 != NONE64 ? order_key(key_value(a1) + key_value(a2)) : a1;
        if (p.whole) g = __shfl_sync(FULL, g, lane << p.lsh & 31);
        if (lane >= p.G) g = NONE64;
        const unsigned keep = kept_groups<long long>(p, lane, g);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int at = (lane * VPL + i) / p.gs;
            if (at >= p.G || !((keep >> at) & 1u)) {
                c[i] = -CUDART_INF_F;
                h[i] = NONE64;
            }
        }
    }
    {
        // near a taken rank other than its own, or near the last
        const int key = take_rough<VPL>(c, lane, p.K);
        const float v = key >= FIRST ? key_value(key & ~255) : -CUDART_INF_F;
        const float last = __shfl_sync(FULL, v, p.K - 1);
        int n[VPL] = {};
        for (int k = 0; k < p.K; ++k) {
            const float vk = __shfl_sync(FULL, v, k), sk = 2.0f * slack(vk);
#pragma unroll
            for (int i = 0; i < VPL; ++i) n[i] += fabsf(c[i] - vk) <= sk || c[i] == vk ? 1 : 0;
        }
        unsigned need = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (c[i] > -CUDART_INF_F && (n[i] >= 2 || fabsf(c[i] - last) <= 2.0f * slack(last) || c[i] == last)) need |= 1u << i;
        make_exact(need);
    }
    int id = -1;
    for (int k = 0; k < p.K; ++k) {
        long long best = h[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < VPL; ++i)
            if (h[i] > best) {
                best = h[i];
                at = i;
            }
        const int hi = __reduce_max_sync(FULL, static_cast<int>(best >> 32));
        const bool top = static_cast<int>(best >> 32) == hi;
        const unsigned lo = __reduce_max_sync(FULL, top ? static_cast<unsigned>(best) : 0u);
        const int from = __ffs(__ballot_sync(FULL, top && static_cast<unsigned>(best) == lo)) - 1;
        if (hi == static_cast<int>(NONE64 >> 32) && lo == 0u) break;
        const int e = __shfl_sync(FULL, lane * VPL + at, from);
        if (lane == k) id = e;
        if (lane == from) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i == at) h[i] = NONE64;
        }
    }
    write_token(p, t, lane, id, id >= 0 ? clean(to_f32(row[id])) : -CUDART_INF_F, m, z, idx, w);
}

template <int VPL, typename T, bool VEC>
__global__ void __launch_bounds__(32 * WARPS, 8)
group_route_kernel(const __grid_constant__ Params p, const T* __restrict__ logits, int32_t* __restrict__ idx,
                   float* __restrict__ w) {
    __shared__ float copies[WARPS][32 * VPL];
    const int lane = static_cast<int>(lane_id());
    float* copy = copies[threadIdx.x >> 5];
    pdl_wait();
    pdl_trigger();
    const int step = gridDim.x * WARPS;
    const int t0 = blockIdx.x * WARPS + (threadIdx.x >> 5);
    const bool by_logit = p.bias == nullptr;
    // 32 tokens of the warp at a time; the near ones of them follow, in FP64
    for (long long tb = t0; tb < p.T; tb += 32LL * step) {
        unsigned again = 0;  // tokens that FP32 and the short resolutions left open
        float r[VPL], b[VPL];
        load_row<VPL, T, VEC>(logits + tb * p.stride, lane, p.E, r);
        lane_bias<VPL, VEC>(p, lane, b);
        for (int k = 0; k < 32; ++k) {
            const long long t = tb + static_cast<long long>(k) * step;
            if (t >= p.T) break;
            const T* row = logits + t * p.stride;
            float c[VPL], m, z, inv;
            choices<VPL>(p, r, b, c, m, z, inv);
            bool near = false, gnear = false, close = false;
            // How near two FP32 choices may lie before FP64 decides, both sides' errors
            // together and not quite twice what they can be. A sigmoid: 4.4 units of 2^-24
            // (exponential 2^-22 of itself and 1.5 |r| 2^-24 of its argument, both times
            // s (1 - s); sum, reciprocal); a softmax score: 22 + |r - m| units of itself,
            // at most 23 of the largest; the bias's addition: one unit of the choice.
            const float sabs = p.softmax ? 0x1p-18f * inv : 0x1p-20f;
            const bool ranked = by_logit && (p.G == 1 || p.rank == 1);
            if (ranked) logits_rank<VPL>(r, c);
            if (p.G > 1) {
                float lo, hi, mag, mine, a2;
                unsigned keep = choose_groups<VPL>(p, lane, c, copy, lo, hi, mag, mine, a2);
                if (hi > -CUDART_INF_F && p.TG < p.G) {
                    // without a bias a score names its logit: |r| and |r - m| are below 48 from 1e-20 on
                    const float tol = ranked ? logit_slack(p, m, lo, hi)
                                      : p.bias != nullptr ? 2.0f * sabs + 0x1p-22f * mag : 0x1p-15f * lo;
                    gnear = !(lo - hi > tol) || (by_logit && !ranked && lo < 1e-20f);
                    // an exact tie: the lower index stays, unless FP64 knows more equals (not where
                    // even the type's next value is clear)
                    constexpr float STEP = sizeof(T) == 2 ? 0x1p-12f : 0x1p-25f;
                    if (ranked && lo == hi) gnear = !(tol <= STEP * fabsf(lo) && lo < CUDART_INF_F) && tied_border_near(&p, m, mine, lo);
                    if (gnear && !ranked && isfinite(tol) && !(by_logit && lo < 1e-20f))
                        gnear = !choose_groups_exact<T>(&p, row, m, inv, mine, a2, lo, hi, tol, &keep);
                }
                if (p.whole) {
                    const int at = lane >> p.lsh;
                    if (at >= p.G || !((keep >> at) & 1u)) {
#pragma unroll
                        for (int i = 0; i < VPL; ++i) c[i] = -CUDART_INF_F;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < VPL; ++i)
                        if (!((keep >> ((lane * VPL + i) * p.per_group >> 16 & 31)) & 1u)) c[i] = -CUDART_INF_F;
                }
            }
            if (by_logit && !ranked) logits_rank<VPL>(r, c);
            if (t + step < p.T) load_row<VPL, T, VEC>(row + step * p.stride, lane, p.E, r);
            // two more than K: the rank behind the last taken one, and one that bounds the rest
            const int key = take_rough<VPL>(c, lane, p.K + 2);
            int id = -1;
            float rk = -CUDART_INF_F, val = -CUDART_INF_F;
            if (key >= FIRST) {
                id = 255 - (key & 255);
                rk = clean(to_f32(row[id]));
                val = by_logit ? rk : choice(p, rk, __ldg(p.bias + id), m, inv);
            }
            // every expert behind lies at or below the last key with its dropped bits set (an
            // infinity stays one); a key drops nothing of a 16-bit logit
            const bool whole = by_logit && sizeof(T) == 2;
            if (!whole && lane > p.K && key >= FIRST) val = key_value(min(key | 255, 0x7f800000));
            const float rest = __shfl_sync(FULL, val, p.K + 1);
            const float next = __shfl_down_sync(FULL, val, 1);
            if (__any_sync(FULL, lane < p.K && next > val)) {
                // ranks that the dropped bits had out of order
                int rank = 0;
                for (int j = 0; j <= p.K; ++j) {
                    const float o = __shfl_sync(FULL, val, j);
                    const int oid = __shfl_sync(FULL, id, j);
                    rank += (o > val || (o == val && oid < id)) ? 1 : 0;
                }
                if (lane > p.K || id < 0) rank = lane;
                int src = lane;
                for (int j = 0; j <= p.K; ++j)
                    if (__shfl_sync(FULL, rank, j) == lane) src = j;
                id = __shfl_sync(FULL, id, src);
                rk = __shfl_sync(FULL, rk, src);
                val = __shfl_sync(FULL, val, src);
            }
            const int id2 = __shfl_down_sync(FULL, id, 1);
            const float val2 = __shfl_down_sync(FULL, val, 1), rk2 = __shfl_down_sync(FULL, rk, 1);
            if (lane < p.K && id2 >= 0) {
                const float tol = by_logit ? logit_slack(p, m, val, val2) : sabs + 0x1p-22f * fabsf(val);
                // equal inputs are an exact tie: the lower index is first already
                if (!(val - val2 > tol)) close = !(rk == rk2 && (by_logit || p.bias[id] == p.bias[id2]));
                near = lane == p.K - 1 && rest > -CUDART_INF_F && !(val - rest > tol);
                // whole keys rank equal logits; the next lower one is a step of the type below, and
                // clear (not below an infinity, whose sigmoid large logits have in FP64 too)
                if (whole && rest == val && val < CUDART_INF_F && tol <= 0x1p-12f * fabsf(val)) near = false;
            }
            near = near || gnear;
            if (__any_sync(FULL, close)) {
                if (__any_sync(FULL, near) || (p.softmax && !by_logit)) near = true;
                else order_exact(p, lane, m, by_logit || id < 0 ? 0.0f : p.bias[id], id, rk);
            }
            if (__any_sync(FULL, near)) again |= 1u << k;
            else write_token(p, t, lane, id, rk, m, z, idx, w);
        }
        for (; again; again &= again - 1) {
            const long long t = tb + static_cast<long long>(__ffs(again) - 1) * step;
            route_exact<VPL, T, VEC>(&p, t, logits + t * p.stride, idx, w);
        }
    }
}

// dL/dr of L = sum dw w with the selection held fixed. With q = s / sum s over
// the selected and v = sum dw q:
//   renormalised softmax  dr_k = scale q_k (dw_k - v), zero off the selection
//   renormalised sigmoid  the same times 1 - s_k
//   raw sigmoid           dr_k = scale dw_k s_k (1 - s_k)
//   raw softmax           dr_e = s_e (scale [e taken] dw_e - sum_k scale dw_k s_k)
// Only the last reads the logits off the selection.
template <int VPL, typename T, bool VEC>
__global__ void __launch_bounds__(32 * WARPS)
group_route_bwd_kernel(Params p, const T* __restrict__ logits, const int32_t* __restrict__ idx,
                       const float* __restrict__ dw, T* __restrict__ dr) {
    __shared__ float srow[WARPS][32 * VPL + VPL];
    const int lane = static_cast<int>(lane_id());
    float* u = srow[threadIdx.x >> 5];
    pdl_wait();
    pdl_trigger();
    const int step = gridDim.x * WARPS;
    const bool dense = p.softmax && !p.renorm;
    for (int t = blockIdx.x * WARPS + (threadIdx.x >> 5); t < p.T; t += step) {
        const T* row = logits + t * p.stride;
        float r[VPL], m = 0.0f, z = 1.0f, e[VPL];
        int id = -1;
        float g = 0.0f, rk = -CUDART_INF_F;
        if (lane < p.K) {
            id = idx[static_cast<long long>(t) * p.K + lane];
            if (id >= 0 && id < p.E) {
                rk = clean(to_f32(row[id]));
                g = p.scale * dw[static_cast<long long>(t) * p.K + lane];
            }
        }
        // a masked expert among the given ids has score 0: no gradient passes
        const bool there = lane < p.K && id >= 0 && id < p.E && rk > -CUDART_INF_F;
        if (dense) {
            load_row<VPL, T, VEC>(row, lane, p.E, r);
            float mx = r[0];
#pragma unroll
            for (int i = 1; i < VPL; ++i) mx = fmaxf(mx, r[i]);
            m = warp_max(mx);
            z = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                e[i] = r[i] == -CUDART_INF_F ? 0.0f : r[i] == m ? 1.0f : expf(r[i] - m);
                z += e[i];
            }
            z = warp_add(z);
            if (z == 0.0f) z = 1.0f;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) u[lane * VPL + i] = 0.0f;
        float q;
        const float s = selected_score(p, there, rk, m, z, q);
        const float v = warp_add(there ? g * (p.renorm ? q : s) : 0.0f);
        float d = g;
        if (!dense) {
            if (p.renorm) d = q * (g - v);
            if (!p.softmax) {
                const float ex = expf(-fabsf(rk)), rest = rk >= 0.0f ? ex / (1.0f + ex) : 1.0f / (1.0f + ex);
                d = (p.renorm ? d : g * s) * rest;
            }
        }
        __syncwarp();
        if (there) u[id] = d;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int ex = lane * VPL + i;
            r[i] = u[ex];
            if (dense) r[i] = e[i] / z * (r[i] - v);
        }
        T* out = dr + static_cast<long long>(t) * p.E;
        if constexpr (VEC) {
            if (lane * VPL < p.E) {
                constexpr int B = VPL * sizeof(T) >= 16 ? 16 : VPL * sizeof(T);
                constexpr int N = B / sizeof(T);
#pragma unroll
                for (int i = 0; i < VPL; i += N) {
                    alignas(16) T o[N];
#pragma unroll
                    for (int j = 0; j < N; ++j) o[j] = from_f32<T>(r[i + j]);
                    T* at = out + lane * VPL + i;
                    if constexpr (B == 16)
                        *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(o);
                    else if constexpr (B == 8)
                        *reinterpret_cast<uint2*>(at) = *reinterpret_cast<const uint2*>(o);
                    else if constexpr (B == 4)
                        *reinterpret_cast<uint32_t*>(at) = *reinterpret_cast<const uint32_t*>(o);
                    else
                        at[0] = o[0];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (lane * VPL + i < p.E) out[lane * VPL + i] = from_f32<T>(r[i]);
        }
        __syncwarp();
    }
}

template <int VPL, typename T>
cudaError_t launch_t(const GroupRouteArgs& a, Params p, bool bwd, cudaStream_t s) {
    const int want = (a.T + WARPS - 1) / WARPS, cap = num_sms() * (bwd ? 16 : 32);
    const dim3 grid(want < cap ? want : cap), block(32 * WARPS);
    // vector rows: every lane's run of experts whole and aligned
    constexpr int B = VPL * static_cast<int>(sizeof(T)) >= 16 ? 16 : VPL * static_cast<int>(sizeof(T));
    auto even = [&](const void* q, long long st) {
        return reinterpret_cast<uintptr_t>(q) % B == 0 && st * static_cast<long long>(sizeof(T)) % B == 0;
    };
    const bool vec = a.E % VPL == 0 && even(a.logits, a.stride) && (!bwd || even(a.dlogits, a.E)) &&
                     reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    const T* lg = static_cast<const T*>(a.logits);
    if (!bwd)
        return vec ? launch_pdl(group_route_kernel<VPL, T, true>, grid, block, 0, s, p, lg, a.idx, a.w)
                   : launch_pdl(group_route_kernel<VPL, T, false>, grid, block, 0, s, p, lg, a.idx, a.w);
    const int32_t* ci = a.idx;
    T* dl = static_cast<T*>(a.dlogits);
    return vec ? launch_pdl(group_route_bwd_kernel<VPL, T, true>, grid, block, 0, s, p, lg, ci, a.dw, dl)
               : launch_pdl(group_route_bwd_kernel<VPL, T, false>, grid, block, 0, s, p, lg, ci, a.dw, dl);
}

template <typename T>
cudaError_t launch_d(const GroupRouteArgs& a, bool bwd, cudaStream_t s) {
    Params p{};
    p.T = a.T;
    p.E = a.E;
    p.K = a.K;
    p.G = a.G;
    p.gs = a.E / a.G;
    p.TG = a.TG;
    p.rank = a.rank;
    p.softmax = a.softmax;
    p.renorm = a.renorm;
    p.scale = a.scale;
    p.stride = a.stride;
    p.bias = a.bias;
    const int vpl = a.E <= 32 ? 1 : a.E <= 64 ? 2 : a.E <= 128 ? 4 : 8;
    const int lg = p.gs % vpl == 0 ? p.gs / vpl : 0;
    p.whole = lg > 0 && (lg & (lg - 1)) == 0;
    while ((p.whole ? lg : 32 / p.G) >> (p.lsh + 1)) ++p.lsh;
    p.lg = 1 << p.lsh;
    p.per_group = (65536 + p.gs - 1) / p.gs;
    if (vpl == 1) return launch_t<1, T>(a, p, bwd, s);
    if (vpl == 2) return launch_t<2, T>(a, p, bwd, s);
    if (vpl == 4) return launch_t<4, T>(a, p, bwd, s);
    return launch_t<8, T>(a, p, bwd, s);
}

}  // namespace

cudaError_t launch_group_route(const GroupRouteArgs& a, bool bwd, cudaStream_t s) {
    switch (a.dtype) {
        case MOE_BF16: return launch_d<__nv_bfloat16>(a, bwd, s);
        case MOE_F16: return launch_d<__half>(a, bwd, s);
        default: return launch_d<float>(a, bwd, s);
    }
}

}  // namespace moe
