// C entry points of the operators around the layer (declared in
// include/moe.h): layer norm, group-limited routing, row quantisation and the
// 8-bit expert products. Host-side validation, then the launchers.
#include <math.h>
#include <stdlib.h>

#include "common.cuh"
#include "internal.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

using namespace moe;

namespace {

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool known_dtype(int32_t t) { return t == MOE_F32 || t == MOE_BF16 || t == MOE_F16; }
size_t elem_size(int32_t t) { return t == MOE_F32 ? 4 : 2; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Rows, row length, type and row pitch shared by the row operators.
moe_status check_rows(int32_t R, int32_t d, int32_t dtype, int64_t stride) {
    if (R < 0 || d < 1 || !known_dtype(dtype) || stride < 0) return MOE_ERR_INVALID_ARG;
    if (R > 1 && stride < d) return MOE_ERR_INVALID_ARG;
    if (d > (1 << 24) || R > (1 << 30)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

MOE_API moe_status moe_layer_norm(int32_t R, int32_t d, int32_t dtype, const void* x, int64_t x_stride,
                                  const float* gamma, const float* beta, float eps, void* y, int64_t y_stride,
                                  float* mean, float* rstd, void* stream) {
    moe_status v = check_rows(R, d, dtype, x_stride);
    if (v == MOE_OK) v = check_rows(R, d, dtype, y_stride);
    if (v != MOE_OK) return v;
    if (!(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
    if (R == 0) return MOE_OK;
    if (!x || !y || !aligned(x, elem_size(dtype)) || !aligned(y, elem_size(dtype)) || !aligned(gamma, 4) ||
        !aligned(beta, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
        return MOE_ERR_INVALID_ARG;
    LayerNormArgs a{};
    a.R = R; a.d = d; a.dtype = dtype;
    a.x = x; a.x_stride = x_stride;
    a.gamma = gamma; a.beta = beta; a.eps = eps;
    a.y = y; a.y_stride = y_stride;
    a.mean_out = mean; a.rstd_out = rstd;
    return cuda_status(launch_layer_norm(a, static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status moe_layer_norm_backward_workspace_size(int32_t R, int32_t d, size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status v = check_rows(R, d, MOE_F32, d);
    if (v != MOE_OK) return v;
    *bytes = R == 0 ? 0 : static_cast<size_t>(layer_norm_bwd_parts(R, d)) * 2 * static_cast<size_t>(d) * 4;
    return MOE_OK;
}

MOE_API moe_status moe_layer_norm_backward(int32_t R, int32_t d, int32_t dtype, const void* dy, int64_t dy_stride,
                                           const void* x, int64_t x_stride, const float* mean, const float* rstd,
                                           const float* gamma, void* dx, int64_t dx_stride, float* dgamma,
                                           float* dbeta, void* ws, size_t ws_bytes, void* stream) {
    moe_status v = check_rows(R, d, dtype, dy_stride);
    if (v == MOE_OK) v = check_rows(R, d, dtype, x_stride);
    if (v == MOE_OK) v = check_rows(R, d, dtype, dx_stride);
    if (v != MOE_OK) return v;
    const size_t es = elem_size(dtype);
    if (!aligned(dgamma, 4) || !aligned(dbeta, 4)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (R == 0) {  // sums over no rows
        if (dgamma && cudaMemsetAsync(dgamma, 0, static_cast<size_t>(d) * 4, s) != cudaSuccess) return MOE_ERR_CUDA;
        if (dbeta && cudaMemsetAsync(dbeta, 0, static_cast<size_t>(d) * 4, s) != cudaSuccess) return MOE_ERR_CUDA;
        return MOE_OK;
    }
    if (!dy || !x || !mean || !rstd || !dx || !aligned(dy, es) || !aligned(x, es) || !aligned(dx, es) ||
        !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(gamma, 4))
        return MOE_ERR_INVALID_ARG;
    const bool cols = dgamma != nullptr || dbeta != nullptr;
    if (cols) {
        size_t need = 0;
        moe_layer_norm_backward_workspace_size(R, d, &need);
        if (!ws || !aligned(ws, 16)) return MOE_ERR_INVALID_ARG;
        if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    }
    LayerNormArgs a{};
    a.R = R; a.d = d; a.dtype = dtype;
    a.x = x; a.x_stride = x_stride;
    a.dy = dy; a.dy_stride = dy_stride;
    a.mean = mean; a.rstd = rstd; a.gamma = gamma;
    a.y = dx; a.y_stride = dx_stride;
    a.dgamma = dgamma; a.dbeta = dbeta;
    return cuda_status(launch_layer_norm_bwd(a, cols ? static_cast<float*>(ws) : nullptr, s));
}

namespace {

moe_status check_group_route(const moe_group_route_config& c, int64_t stride) {
    if (c.T < 0 || c.E < 1 || c.K < 1 || c.K > c.E || !known_dtype(c.dtype)) return MOE_ERR_INVALID_ARG;
    if (c.score != MOE_SCORE_SIGMOID && c.score != MOE_SCORE_SOFTMAX) return MOE_ERR_INVALID_ARG;
    if (c.renormalize != 0 && c.renormalize != 1) return MOE_ERR_INVALID_ARG;
    if (!(c.scale == c.scale)) return MOE_ERR_INVALID_ARG;
    if (c.n_groups < 1 || c.E % c.n_groups || c.topk_groups < 1 || c.topk_groups > c.n_groups)
        return MOE_ERR_INVALID_ARG;
    if (c.group_rank != 1 && c.group_rank != 2) return MOE_ERR_INVALID_ARG;
    if (c.K > c.E / c.n_groups * c.topk_groups) return MOE_ERR_INVALID_ARG;
    if (stride < 0 || (c.T > 1 && stride < c.E)) return MOE_ERR_INVALID_ARG;
    if (c.E > 256 || c.K > 16 || c.n_groups > 32 || c.T > (1 << 30)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

GroupRouteArgs group_args(const moe_group_route_config& c, const void* logits, int64_t stride) {
    GroupRouteArgs a{};
    a.T = c.T; a.E = c.E; a.K = c.K; a.G = c.n_groups; a.TG = c.topk_groups; a.rank = c.group_rank;
    a.softmax = c.score == MOE_SCORE_SOFTMAX; a.renorm = c.renormalize; a.dtype = c.dtype;
    a.scale = c.scale; a.logits = logits; a.stride = stride;
    return a;
}

}  // namespace

MOE_API moe_status moe_group_route(const moe_group_route_config* cfg, const void* logits, int64_t row_stride,
                                   const float* bias, int32_t* topk_idx, float* topk_w, void* stream) {
    if (!cfg) return MOE_ERR_INVALID_ARG;
    const moe_status v = check_group_route(*cfg, row_stride);
    if (v != MOE_OK || cfg->T == 0) return v;
    if (!logits || !topk_idx || !topk_w || !aligned(logits, elem_size(cfg->dtype)) || !aligned(bias, 4) ||
        !aligned(topk_idx, 4) || !aligned(topk_w, 4))
        return MOE_ERR_INVALID_ARG;
    GroupRouteArgs a = group_args(*cfg, logits, row_stride);
    a.bias = bias; a.idx = topk_idx; a.w = topk_w;
    return cuda_status(launch_group_route(a, false, static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status moe_group_route_backward(const moe_group_route_config* cfg, const void* logits,
                                            int64_t row_stride, const int32_t* topk_idx, const float* dw,
                                            void* dlogits, void* stream) {
    if (!cfg) return MOE_ERR_INVALID_ARG;
    const moe_status v = check_group_route(*cfg, row_stride);
    if (v != MOE_OK || cfg->T == 0) return v;
    const size_t es = elem_size(cfg->dtype);
    if (!logits || !topk_idx || !dw || !dlogits || !aligned(logits, es) || !aligned(dlogits, es) ||
        !aligned(topk_idx, 4) || !aligned(dw, 4))
        return MOE_ERR_INVALID_ARG;
    GroupRouteArgs a = group_args(*cfg, logits, row_stride);
    a.idx = const_cast<int32_t*>(topk_idx); a.dw = dw; a.dlogits = dlogits;
    return cuda_status(launch_group_route(a, true, static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status moe_quantize_rows(int32_t R, int32_t K, int32_t dtype, const void* x, int64_t x_stride,
                                     int8_t* q, float* scale, void* stream) {
    const moe_status v = check_rows(R, K, dtype, x_stride);
    if (v != MOE_OK || R == 0) return v;
    if (!x || !q || !scale || !aligned(x, elem_size(dtype)) || !aligned(scale, 4)) return MOE_ERR_INVALID_ARG;
    QuantArgs a{R, K, dtype, x, x_stride, q, scale};
    return cuda_status(launch_quantize_rows(a, static_cast<cudaStream_t>(stream)));
}

namespace {

moe_status check_int8(const moe_int8_config& c) {
    if (c.M < 0 || c.Ma < 0 || c.K < 1 || c.N < 1 || c.E < 1 || !known_dtype(c.out_dtype)) return MOE_ERR_INVALID_ARG;
    if (c.swiglu != 0 && c.swiglu != 1) return MOE_ERR_INVALID_ARG;
    if (c.swiglu && c.N % 2) return MOE_ERR_INVALID_ARG;
    // 16-byte rows of 8-bit values; the largest sum, K 2^14, fits 32 bits
    if (c.K % 16 || c.K > 131056 || c.E > 256 || c.N > (1 << 24) || c.M > (1 << 30)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// The form of a product, from sizes alone. MOE_INT8_FORM overrides the choice
// for tests and tuning.
//   Integer dot products while the whole product is small, or few experts have rows:
//   they have no tokens' pass and spread over channels (us, dot products against tiles
//   of 32: one row, 4096 x 2048, 8 : 25; 16 rows, 4096 x 4096, 16 : 29; 16 rows,
//   4096 x 16384, 45 : 33; 128 rows of 64 experts, 2048 x 1408, 49 : 47; 64 rows of 256
//   experts, 4096 x 4096, 150 : 174; 128, 279 : 291; 256, 469 : 434). A step of their
//   reduction is 512 values, whatever part of it is there.
//   Tiles of 32 rows while they hold an expert's (against 256: 2 rows each of 256
//   experts, 4096 x 4096, 571 : 701; 4 each, 645 : 787).
//   Else the form whose waves take less: one of 32-row tiles on every SM takes 1.2 us
//   and 3.2 ns a reduction step, one of 256-row tiles on the pairs 3 us and 4.5 ns, and
//   4 us more to begin (tiles of 32 against 256: 801 rows, 368 x 574, 12 : 18; 128 rows,
//   4096 x 4096, 29 : 35; 4096 x 16384, 66 : 39; 160 rows, 8192 x 2048, 47 : 61;
//   4000 rows, 256 x 1024, 20 : 18; 10676 rows of 4, 3440 x 245, 80 : 51).
enum Int8Form { INT8_VEC, INT8_SMALL, INT8_WIDE };
Int8Form int8_form(const moe_int8_config& c) {
    if (const char* e = getenv("MOE_INT8_FORM")) {
        if (e[0] == 'v') return INT8_VEC;
        if (e[0] == 's') return INT8_SMALL;
        if (e[0] == 'w') return INT8_WIDE;
    }
    const double steps = static_cast<double>(c.M) * c.N * ((c.K + 511) / 512 * 512);
    if (c.M <= 32LL * c.E && (2LL * c.M <= c.E || steps <= 268435456.0)) return INT8_VEC;
    if (c.M <= 32LL * c.E) return INT8_SMALL;
    const int F = c.swiglu ? c.N / 2 : c.N, sms = num_sms();
    // us of tiles of `rows` rows and `chans` outputs, at most one part full an expert
    auto waves = [&](int rows, int chans, int at_a_time, double us, double us_per_k) {
        const double tiles = ((c.M + rows - 1) / rows + (c.E > 1 ? c.E : 0)) * static_cast<double>((F + chans - 1) / chans);
        return ceil(tiles / at_a_time) * (us + us_per_k * c.K);
    };
    const double small = waves(32, c.swiglu ? 64 : 128, sms, 1.2, 3.2e-3);
    return small <= 4.0 + waves(256, c.swiglu ? 128 : 256, sms / 2, 3.0, 4.5e-3) ? INT8_SMALL : INT8_WIDE;
}

}  // namespace

MOE_API moe_status moe_matmul_int8_workspace_size(const moe_int8_config* cfg, size_t* bytes) {
    if (!cfg || !bytes) return MOE_ERR_INVALID_ARG;
    const moe_status v = check_int8(*cfg);
    if (v != MOE_OK) return v;
    *bytes = cfg->M == 0 ? 0 : int8_tc_workspace(cfg->M, cfg->K);  // whichever form the call takes
    return MOE_OK;
}

MOE_API moe_status moe_matmul_int8(const moe_int8_config* cfg, const int8_t* a, int64_t a_stride,
                                   const float* a_scale, const int8_t* b, const float* b_scale,
                                   const int32_t* offsets, const int32_t* rows, void* out, void* ws,
                                   size_t ws_bytes, void* stream) {
    if (!cfg) return MOE_ERR_INVALID_ARG;
    const moe_status v = check_int8(*cfg);
    if (v != MOE_OK) return v;
    const moe_int8_config& c = *cfg;
    if (!offsets && c.E != 1) return MOE_ERR_INVALID_ARG;
    if (!rows && c.M > c.Ma) return MOE_ERR_INVALID_ARG;
    if (c.M == 0) return MOE_OK;
    if (c.Ma == 0) return MOE_ERR_INVALID_ARG;
    if (a_stride < 0 || (c.Ma > 1 && a_stride < c.K) || a_stride % 16) return MOE_ERR_INVALID_ARG;
    if (!a || !a_scale || !b || !b_scale || !out || !aligned(a, 16) || !aligned(b, 16) || !aligned(out, 16) ||
        !aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(offsets, 4) || !aligned(rows, 4))
        return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    moe_matmul_int8_workspace_size(cfg, &need);
    if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    Int8Args g{};
    g.M = c.M; g.Ma = c.Ma; g.K = c.K; g.N = c.N; g.E = c.E; g.swiglu = c.swiglu; g.out_dtype = c.out_dtype;
    g.lda = a_stride;
    g.a = a; g.sa = a_scale; g.b = b; g.sb = b_scale;
    g.offsets = offsets; g.rows = rows; g.out = out;
    g.err = static_cast<int*>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Int8Form f = int8_form(c);
    return cuda_status(f == INT8_VEC ? launch_int8_vec(g, s) : launch_int8_tc(g, f == INT8_WIDE, s));
}
