/*
 * moe.h - C ABI of the GB300 (sm_103a) forward (and backward) pass of a
 * top-K routed Mixture-of-Experts SwiGLU FFN layer with always-on shared
 * experts.
 *
 * The layer (APEX-1 Mathematical Reference Part 3, section 13.2):
 *
 *     MoE(x) = sum_{s<S} Shared_s(x) + sum_{k<K} g_k * Expert_{e_k}(x)
 *     Expert(x) = W_down( SiLU(x W_gate) (.) x W_up )          (section 12.2)
 *
 * with router logits r = x W_router in FP32, an optional per-expert balance
 * bias, top-K selection and one of three gate rules (see moe_gate). In the
 * latent variant (kimi_k3 "StableLatentMoE and QuantileBalancer") the routed
 * experts act on z = x W_down_latent and their weighted sum is projected back
 * by W_up_latent before the shared output is added.
 *
 * Conventions for every entry point:
 *  - Every array is row-major and contiguous. "Device" pointers must point to
 *    memory of the current CUDA device; "host" pointers to host memory.
 *  - The caller owns every buffer. The library allocates no device memory;
 *    scratch space is the caller's workspace (see moe_workspace_size).
 *  - Work is enqueued on the given stream (a cudaStream_t passed as void*,
 *    NULL = the legacy default stream) and the call returns without
 *    synchronising, except where a function says otherwise.
 *  - Arguments are validated on the host before anything is launched; an
 *    invalid call returns an error code and enqueues nothing.
 *  - Expert ids are int32; FP32 is IEEE binary32; BF16 is bfloat16 (the
 *    upper 16 bits of a binary32), rounded to nearest-even where produced.
 *  - No entry point is thread-safe with respect to a workspace: concurrent
 *    calls must use distinct workspaces.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misaligned pointer, K > E, ... */
    MOE_ERR_UNSUPPORTED = 2,  /* valid but outside what the kernels implement (e.g. E > 256) */
    MOE_ERR_WORKSPACE = 3,    /* workspace smaller than moe_workspace_size() */
    MOE_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
    MOE_ERR_TIMEOUT = 5,      /* a device-side wait ran out of time (see moe_workspace_status) */
    MOE_ERR_DEVICE_INDEX = 6  /* a kernel met an expert id outside [0, E) */
} moe_status;

typedef enum moe_dtype {
    MOE_F32 = 0,   /* FP32 activations and expert weights, FP32 FMA arithmetic */
    MOE_BF16 = 1,  /* BF16 activations and expert weights, FP32 accumulation (tcgen05) */
    MOE_F16 = 2    /* FP16 (IEEE binary16): the operators around the layer only (moe_layer_norm
                      and what follows it below); a moe_config refuses it */
} moe_dtype;

/* Gate rule. c denotes the selection score, b the balance bias.
 * Top-K ranks by c descending; equal scores rank the lower expert id first;
 * slot k of every [T, K] output holds the k-th ranked expert. */
typedef enum moe_gate {
    /* c = r + b; top-K of c; g = softmax over the K selected c.
     * (APEX-1 docs "10 - Mixture of Experts", MoEFFN.forward steps 2-3;
     *  APEX-1 Math Ref Part 3 section 13.2) */
    MOE_GATE_SOFTMAX_TOPK = 0,
    /* p = softmax over all E of (r + b); c = p; top-K of p; g = p_sel / sum p_sel.
     * ("MoE from scratch" tutorial, MoELayer.forward) */
    MOE_GATE_SOFTMAX_ALL_RENORM = 1,
    /* s = sigmoid(r); c = s + b; top-(K+1) of c, the first K used; g = s at the
     * selected experts (uncorrected), divided by its sum if renormalize, times
     * routed_scale. (kimi_k3 StableLatentMoE, "FP32 router and training-only QB
     * update", "Flatten routing and recover original token order") */
    MOE_GATE_SIGMOID = 2
} moe_gate;

/* Problem description. */
typedef struct moe_config {
    int32_t T;            /* tokens (batch x sequence flattened), >= 1 */
    int32_t d;            /* model width (M of the latent page) */
    int32_t d_ff;         /* routed expert hidden width (I of the latent page) */
    int32_t E;            /* routed experts, 1..256 */
    int32_t K;            /* active experts per token, 1..min(E,16); K+1 <= E in sigmoid mode */
    int32_t n_shared;     /* always-on shared experts S >= 0 */
    int32_t shared_d_ff;  /* hidden width of each shared expert */
    int32_t latent_dim;   /* 0: experts act on x; L > 0: experts act on z = x W_down_latent */
    int32_t dtype;        /* moe_dtype of x, out and every expert/shared/latent weight */
    int32_t gate;         /* moe_gate */
    int32_t renormalize;  /* sigmoid mode: divide the K weights by their sum */
    float routed_scale;   /* sigmoid mode: factor on the routed weights (1.0 = none) */
    int32_t out_dtype;    /* moe_dtype of out: MOE_F32 (the FP32 accumulation, unrounded) or
                             MOE_BF16 (rounded once to nearest-even); must be MOE_F32 when
                             dtype is MOE_F32 */
    int32_t save_gate_up; /* 0 or 1. 1, for a layer whose moe_backward runs on the tensor
                             cores (BF16, widths multiples of 64): moe_forward also keeps
                             the gate and up products a = z W_gate, u = z W_up of every
                             routed row and shared expert (BF16) in the workspace, and
                             moe_backward reads them instead of recomputing them (the
                             workspace grows by 4 (T K d_ff + T n_shared shared_d_ff)
                             bytes). The forward and the backward of one step must use the
                             same value. Ignored by other layers. */
} moe_config;

/* Weights, all device pointers. d_e = latent_dim ? latent_dim : d.
 * W_router  [d, E] FP32                       (always FP32, always read as FP32)
 * bias      [E]   FP32, or NULL for no bias
 * W_gate    [E, d_e, d_ff]  W_up [E, d_e, d_ff]  W_down [E, d_ff, d_e]      (dtype)
 * Ws_gate   [S, d, shared_d_ff]  Ws_up [S, d, shared_d_ff]
 * Ws_down   [S, shared_d_ff, d]                                              (dtype)
 * W_down_latent [d, L], W_up_latent [L, d]   (dtype; NULL unless latent_dim > 0)
 * Matrices multiply row vectors from the right: h = x W_gate, y = h W_down. */
typedef struct moe_weights {
    const float* W_router;
    const float* bias;
    const void* W_gate;
    const void* W_up;
    const void* W_down;
    const void* Ws_gate;
    const void* Ws_up;
    const void* Ws_down;
    const void* W_down_latent;
    const void* W_up_latent;
} moe_weights;

/* Device pointers into a workspace after moe_forward: the routing and
 * dispatch results of the last forward that used the workspace. */
typedef struct moe_workspace_views {
    int32_t* topk_idx;      /* [T, K]   selected experts, slot order */
    float* topk_w;          /* [T, K]   gate weights */
    float* margin;          /* [T]      c at rank K minus c at rank K+1 (+inf if K == E) */
    float* top_scores;      /* [T, K+1] sigmoid mode: the K+1 largest c, descending; else NULL */
    float* scores;          /* [T, E]   sigmoid mode: s = sigmoid(r); else NULL */
    int32_t* counts;        /* [E]      assignments per expert */
    int32_t* offsets;       /* [E+1]    exclusive prefix sum of counts */
    int32_t* sorted_token;  /* [T*K]    token of each expert-sorted assignment */
    float* sorted_w;        /* [T*K]    gate weight of each expert-sorted assignment */
    int32_t* inv;           /* [T, K]   sorted position of assignment (t, k) */
} moe_workspace_views;

/* Human-readable name of a status code (static storage). */
const char* moe_status_string(moe_status s);

/* Library version, e.g. "0.1.0" (static storage). */
const char* moe_version(void);

/* Bytes of device workspace moe_forward / moe_dispatch /
 * moe_quantile_bias_update need for cfg (host only, no CUDA call).
 * Returns MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED for an invalid config. */
moe_status moe_workspace_size(const moe_config* cfg, size_t* bytes);

/* Pointers to the routing/dispatch results inside a workspace of cfg
 * (host only; NULL members where the mode has no such array). */
moe_status moe_get_workspace_views(const moe_config* cfg, void* ws, moe_workspace_views* v);

/* Router: logits r = x W_router in FP32 (x read as FP32 when dtype is BF16,
 * which is exact), the mode's selection score, top-K (top-(K+1) in sigmoid
 * mode) and gate weights.
 *   x [T, d] (dtype), W_router [d, E] FP32, bias [E] FP32 or NULL.
 *   Outputs (device): topk_idx [T, K] int32, topk_w [T, K] FP32, required;
 *   margin [T] FP32, top_scores [T, K+1] FP32 and scores [T, E] FP32 optional
 *   (NULL = not written); top_scores/scores are only produced in sigmoid mode.
 *   ws: NULL, or a workspace of moe_workspace_size(cfg) bytes. With a
 *   workspace, BF16 layers with E > 32, E % 8 == 0 and d % 64 == 0 compute
 *   the logits on the tensor cores from an exact three-part BF16 split of
 *   W_router (the same path moe_forward takes); otherwise, and without a
 *   workspace, one fused FP32 FMA kernel computes them. Both are FP32-accurate
 *   but sum in different orders, so near-tie tokens may rank differently.
 * Sources: APEX-1 docs "10 - Mixture of Experts" steps 2-3; APEX-1 Math Ref
 * Part 3 sections 13.2 and 13.5; "MoE from scratch" MoELayer.forward;
 * kimi_k3 StableLatentMoE "FP32 router and training-only QB update". */
moe_status moe_route(const moe_config* cfg, const void* x, const float* W_router,
                     const float* bias, int32_t* topk_idx, float* topk_w, float* margin,
                     float* top_scores, float* scores, void* ws, size_t ws_bytes, void* stream);

/* Sorted dispatch of the T*K assignments by expert id: a stable counting sort
 * of the flat assignments j = t*K + k (kimi_k3 StableLatentMoE, "Flatten
 * routing and recover original token order" and "Dispatch is a stable
 * permutation").
 *   topk_idx [T, K] int32 (device), topk_w [T, K] FP32 (device).
 *   Outputs (device): counts [E], offsets [E+1] (exclusive prefix sums,
 *   offsets[E] = T*K), sorted_token [T*K] (= j / K of the assignment at each
 *   sorted position), sorted_w [T*K], inv [T, K] (sorted position of (t, k)).
 *   ws: device workspace of at least moe_workspace_size(cfg) bytes.
 * No host synchronisation. An expert id outside [0, E) is skipped and
 * recorded in the workspace (moe_workspace_status returns MOE_ERR_DEVICE_INDEX). */
moe_status moe_dispatch(const moe_config* cfg, const int32_t* topk_idx, const float* topk_w,
                        int32_t* counts, int32_t* offsets, int32_t* sorted_token,
                        float* sorted_w, int32_t* inv, void* ws, size_t ws_bytes,
                        void* stream);

/* moe_dispatch for callers that cannot allocate device memory: for example a
 * runtime that owns all device memory and only hands out the tensors it
 * manages, or code that must not call cudaMalloc after start-up because an
 * allocation can synchronise the device or fail under memory pressure.
 * The pages have no counterpart of this call; it exists for such callers.
 * Same inputs, outputs and results as moe_dispatch, but no workspace: its
 * scratch is a fixed array in the library's own device memory, sized for
 * T*K <= 65536 and E <= 256 (about 130 KB, held by every GPU that loads the
 * library until the process exits); larger calls return MOE_ERR_UNSUPPORTED.
 * The first call on each device looks up the array's device address with
 * that device current; make that first call before any stream capture. The
 * address is kept per device and context: after cudaDeviceReset (or anything
 * else that makes a new context) the next call looks it up again, so make
 * that call before any capture too.
 * Every call reuses the same array, so calls that overlap on the GPU (for
 * example on two streams with no ordering between them) race and corrupt
 * each other's results; order such calls on one stream. Expert ids outside
 * [0, E) are skipped, the other assignments dispatched as moe_dispatch does;
 * the caller detects skipped ids by offsets[E] falling short of T*K by their
 * number. Calls no allocating function. */
moe_status moe_dispatch_noalloc(const moe_config* cfg, const int32_t* topk_idx,
                                const float* topk_w, int32_t* counts, int32_t* offsets,
                                int32_t* sorted_token, float* sorted_w, int32_t* inv,
                                void* stream);

/* Whole layer forward: route -> dispatch -> grouped gate/up GEMM with
 * SiLU(.)*up epilogue -> grouped down GEMM scaled by the gate weight ->
 * shared experts -> deterministic combine (no float atomics).
 *   x [T, d] (dtype, device), out [T, d] (out_dtype, device).
 *   The routing and dispatch results stay in ws (moe_get_workspace_views).
 *   The balance bias is read, never written (use moe_quantile_bias_update).
 *   No host synchronisation and no allocation: after a first call on the
 *   device (which sets kernel attributes), calls can be captured into a CUDA
 *   graph; so can moe_backward.
 *   The grouped GEMMs pick their tile form from the shapes; the environment
 *   variable MOE_GEMM_FORM, read at each call, overrides the choice for tests
 *   and tuning ("rows": row-tile forms only; "single": single-CTA row tiles
 *   only; "tokens": the token-column form wherever the product allows it).
 *   The forms give the same bits except
 *   that the token-column down product stores its routed rows rounded to 16
 *   significant bits (a relative error of at most 2^-17 per routed row).
 * Sources: APEX-1 Math Ref Part 3 sections 12.2 and 13.2; APEX-1 docs
 * "10 - Mixture of Experts" MoEFFN.forward; kimi_k3 StableLatentMoE
 * "Grouped expert execution" and "Return to model width"; "MoE from scratch"
 * MoELayer.forward. */
moe_status moe_forward(const moe_config* cfg, const void* x, const moe_weights* w, void* out,
                       void* ws, size_t ws_bytes, void* stream);

/* moe_forward with HOST input and output: copies x_host [T, d] (dtype) to the
 * device (inside ws), runs the forward and copies out [T, d] (out_dtype) back to
 * out_host, all on `stream`, then synchronises the stream before returning.
 * Pinned host memory makes the copies asynchronous DMA; pageable works too. */
moe_status moe_forward_host(const moe_config* cfg, const void* x_host, const moe_weights* w,
                            void* out_host, void* ws, size_t ws_bytes, void* stream);

/* Quantile balancer update (kimi_k3 "QuantileBalancer: persistent biases, no
 * gradient update"): with p = K/E,
 *     thresh_t = top_scores[t, K]            (the (K+1)-th corrected score)
 *     rel[t, j] = thresh_t - scores[t, j]    (FP32)
 *     b_j = rel[:, j] at sorted index ceil(p (T-1))   ('higher' quantile; the
 *           index computed in FP32 as the FP32 quantile does)
 *     bias = b - mean(b)   (mean: sequential float64 sum over j, divided by E,
 *                           rounded to FP32; FP32 subtraction)
 * Bit-exact for given inputs. top_scores [T, K+1], scores [T, E], bias [E]
 * (output, replaced), all FP32 device. ws: at least moe_workspace_size of a
 * config with the same T, E, K (or moe_quantile_workspace_size bytes). */
moe_status moe_quantile_bias_update(int32_t T, int32_t E, int32_t K, const float* top_scores,
                                    const float* scores, float* bias, void* ws, size_t ws_bytes,
                                    void* stream);

/* Workspace bytes moe_quantile_bias_update needs on its own. */
size_t moe_quantile_workspace_size(int32_t T, int32_t E);

/* Routing diagnostics of one batch: runs the router of cfg on x (as
 * moe_route with a workspace; its selection and logits stay in ws) and
 * writes to out (device, FP32, 2 + E values):
 *     out[0] = aux = E * sum_e f_e P_e      Switch load-balancing loss before
 *                                           its alpha ("MoE from scratch",
 *                                           MoELayer.forward)
 *     out[1] = z = (1/T) sum_t (log sum_e exp r_te)^2   router z-loss before
 *                                           its weight (book-ai MoE chapter,
 *                                           MoELoss.router_z_loss)
 *     out[2 + e] = P_e = (1/T) sum_t softmax(r_t)_e
 * with r = x W_router the raw FP32 logits (no balance bias) and f_e the share
 * of the T*K selected (token, slot) pairs on expert e (the selection uses the
 * bias, as the forward's does). Sums run in a fixed order: the result is
 * reproducible bit for bit. ws: required, at least moe_workspace_size(cfg)
 * bytes, 256-byte aligned; x and W_router 16-byte aligned. */
moe_status moe_routing_stats(const moe_config* cfg, const void* x, const float* W_router,
                             const float* bias, float* out, void* ws, size_t ws_bytes,
                             void* stream);

/* Sign-bias balancing (APEX-1 Math Ref Part 3, section 14.3): with
 * f_e = counts[e] / (N K) and tau = 1/E,
 *     bias[e] <- clamp(bias[e] + alpha * sign(tau - f_e), -1, 1)
 * counts [E] int32 (device, e.g. the workspace's counts after a forward with
 * N = T tokens), bias [E] FP32 device, updated in place. */
moe_status moe_sign_bias_update(int32_t E, int32_t N, int32_t K, const int32_t* counts,
                                float* bias, float alpha, void* stream);

/* Gradients written by moe_backward: FP32 device arrays, row-major. dx is
 * required; any other pointer may be NULL (that gradient is not computed). */
typedef struct moe_grads {
    float* dx;              /* [T, d] */
    float* dW_router;       /* [d, E] */
    float* dW_gate;         /* [E, d_e, d_ff]  d_e = latent_dim ? latent_dim : d */
    float* dW_up;           /* [E, d_e, d_ff] */
    float* dW_down;         /* [E, d_ff, d_e] */
    float* dWs_gate;        /* [S, d, shared_d_ff] */
    float* dWs_up;          /* [S, d, shared_d_ff] */
    float* dWs_down;        /* [S, shared_d_ff, d] */
    float* dW_down_latent;  /* [d, latent_dim] */
    float* dW_up_latent;    /* [latent_dim, d] */
} moe_grads;

/* Bytes of the backward's own scratch workspace (bws of moe_backward). */
moe_status moe_backward_workspace_size(const moe_config* cfg, size_t* bytes);

/* Backward pass: the gradients of L = sum(dout * out) of the forward that
 * last ran on `ws` (moe_forward with the same cfg, x and weights; its routing
 * and dispatch, and for the latent variant z and the routed rows, are read
 * from ws), with that forward's expert selection held fixed - the top-K
 * indices carry no gradient (kimi_k3 StableLatentMoE, "The actual grouped
 * GEMM, and the gradient path"):
 *     gate weights g -> router logits r -> W_router and x, through the gate
 *     rule's formula (the balance bias is a buffer without gradient);
 *     the routed and shared SwiGLU experts, their weights and their input;
 *     the latent projections.
 * Experts that no token selected get no gradient: their slices of dW_gate,
 * dW_up and dW_down are NOT written (kimi_k3 StableLatentMoE, "Grouped
 * expert execution and sparse gradients"); the workspace's counts tell which.
 * Every other requested gradient is overwritten. Sums run in a fixed order:
 * bit-reproducible.
 *   x [T, d] (dtype), dout [T, d] FP32 device; x, dout and every gradient
 *   16-byte aligned.
 * BF16 layers whose d, d_ff, latent_dim and shared_d_ff are multiples of 64
 * run the expert contractions on the tensor cores with BF16 operands (the
 * upstream and activation gradients rounded to BF16, FP32 sums); the others
 * on the CUDA cores in FP32. On the tensor cores, cfg->save_gate_up = 1 takes
 * the gate and up products the forward kept (BF16) instead of recomputing
 * them; the forward must then have run with save_gate_up = 1 as well.
 *   ws: the forward's workspace (moe_workspace_size bytes, 256-byte aligned).
 *   bws: moe_backward_workspace_size bytes, 256-byte aligned. */
moe_status moe_backward(const moe_config* cfg, const void* x, const moe_weights* w,
                        const float* dout, const moe_grads* grads, void* ws, size_t ws_bytes,
                        void* bws, size_t bws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Operators around the layer: the norms around it, group-limited routing, 8-bit
 * expert products and low-rank adapters for serving. Together they make a block
 *   x -> moe_layer_norm -> router logits -> moe_group_route -> moe_dispatch
 *     -> moe_quantize_rows -> moe_matmul_int8 (gate/up, SwiGLU)
 *     -> moe_quantize_rows -> moe_matmul_int8 (down) -> weighted sum per token.
 * Between blocks moe_block_norm joins the residual stream, a block's output and
 * the next block's norm; moe_adapter_add adds the low-rank adapters of many
 * requests to a projection's result.
 * The row operators take rows whose elements are contiguous and whose pitch
 * (`*_stride`, in elements, >= the row's length) is the caller's; zero rows
 * are allowed and launch nothing. Outputs must not overlap inputs. Pointers
 * need their element's alignment; rows on 16-byte boundaries run faster.
 * Each call can be captured into a CUDA graph; results do not depend on the
 * order in which CTAs run.
 * ------------------------------------------------------------------------ */

/* Layer norm of R rows of d elements (d <= 2^24), x and y of type dtype:
 *     mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps)
 *     y  = (x - mu) rstd gamma + beta
 * with FP32 statistics and arithmetic, y rounded once. gamma, beta [d] FP32,
 * either may be NULL (1, 0); mean, rstd [R] FP32 outputs, either may be NULL.
 * eps >= 0. */
moe_status moe_layer_norm(int32_t R, int32_t d, int32_t dtype, const void* x, int64_t x_stride,
                          const float* gamma, const float* beta, float eps, void* y, int64_t y_stride,
                          float* mean, float* rstd, void* stream);

/* Bytes of workspace moe_layer_norm_backward needs where it returns dgamma or
 * dbeta (per-CTA column sums). */
moe_status moe_layer_norm_backward_workspace_size(int32_t R, int32_t d, size_t* bytes);

/* Gradients of L = sum(dy y) given the forward's x, mean and rstd: with
 * xh = (x - mu) rstd and g = dy gamma,
 *     dx = rstd (g - mean(g) - xh mean(g xh)),  dgamma = sum_rows dy xh,
 *     dbeta = sum_rows dy
 * dy, x, dx of type dtype; dgamma, dbeta [d] FP32, overwritten (zeros for
 * R = 0), either may be NULL. ws: 16-byte aligned, needed where one of them
 * is asked for. Sums run in a fixed order: bit-reproducible. */
moe_status moe_layer_norm_backward(int32_t R, int32_t d, int32_t dtype, const void* dy, int64_t dy_stride,
                                   const void* x, int64_t x_stride, const float* mean, const float* rstd,
                                   const float* gamma, void* dx, int64_t dx_stride, float* dgamma,
                                   float* dbeta, void* ws, size_t ws_bytes, void* stream);

typedef enum moe_score {
    MOE_SCORE_SIGMOID = 0,  /* s = sigmoid(r) */
    MOE_SCORE_SOFTMAX = 1   /* s = softmax of r over all E */
} moe_score;

typedef struct moe_group_route_config {
    int32_t T;            /* tokens, >= 0 */
    int32_t E;            /* experts, 1..256 */
    int32_t K;            /* experts taken per token, 1..16, <= topk_groups E / n_groups */
    int32_t n_groups;     /* groups of E / n_groups consecutive experts, 1..32 (1: no groups) */
    int32_t topk_groups;  /* groups kept per token */
    int32_t group_rank;   /* a group's score: 1 = its largest choice, 2 = the sum of its two largest */
    int32_t score;        /* moe_score */
    int32_t renormalize;  /* 0 or 1: divide the K weights by their sum */
    float scale;          /* factor on the weights */
    int32_t dtype;        /* moe_dtype of logits and dlogits */
} moe_group_route_config;

/* Group-limited routing of T rows of E logits: choices c = s + bias, the
 * topk_groups best groups, the K largest c among their experts, weights from
 * the uncorrected s. Equal values rank the lower index first; what is taken
 * is what 64-bit arithmetic on the given logits and bias takes (of a softmax
 * without a bias on its exponentials, whose denominator is common). An expert
 * whose logit or choice is -inf or NaN is never taken: masked experts, and
 * rows that are masked whole, need no other form. Slots without an expert
 * hold id -1 and weight 0 (moe_dispatch skips them and reports
 * MOE_ERR_DEVICE_INDEX). Groups whose experts are all masked rank last.
 *   logits [T, E] (dtype, pitch row_stride), bias [E] FP32 or NULL,
 *   topk_idx [T, K] int32, topk_w [T, K] FP32, slot order by choice. */
moe_status moe_group_route(const moe_group_route_config* cfg, const void* logits, int64_t row_stride,
                           const float* bias, int32_t* topk_idx, float* topk_w, void* stream);

/* Gradient of L = sum(dw topk_w) with respect to the logits, the selection
 * (topk_idx, as moe_group_route gave it: the ids of a row are distinct) held
 * fixed; the bias only chooses and has none. dlogits [T, E] contiguous
 * (dtype) is overwritten; masked experts get 0. Ids outside [0, E) are
 * skipped. */
moe_status moe_group_route_backward(const moe_group_route_config* cfg, const void* logits,
                                    int64_t row_stride, const int32_t* topk_idx, const float* dw,
                                    void* dlogits, void* stream);

/* R rows of K elements to 8-bit integers: scale[i] = max_k |x[i, k]| / 127,
 * q[i, k] = x[i, k] / scale[i] to the nearest integer, ties to even (exactly:
 * the quotient is not rounded first). A row of zeros has scale 0; a row with
 * an infinity or a NaN has q = 0 and scale NaN. q [R, K] contiguous. */
moe_status moe_quantize_rows(int32_t R, int32_t K, int32_t dtype, const void* x, int64_t x_stride,
                             int8_t* q, float* scale, void* stream);

typedef struct moe_int8_config {
    int32_t M;          /* product rows, >= 0 */
    int32_t Ma;         /* rows of a */
    int32_t K;          /* reduction length, a multiple of 16, at most 131056 */
    int32_t N;          /* channels of b per expert */
    int32_t E;          /* experts, 1..256 */
    int32_t swiglu;     /* 1: channels [0, N/2) are gates, [N/2, N) ups, the output SiLU(gate) up */
    int32_t out_dtype;  /* moe_dtype of out */
} moe_int8_config;

/* Bytes of workspace moe_matmul_int8 needs for cfg (0 for M = 0). */
moe_status moe_matmul_int8_workspace_size(const moe_int8_config* cfg, size_t* bytes);

/* 8-bit products with a scale per row of a and per channel of b, grouped by
 * expert: product row i of expert e (offsets[e] <= i < offsets[e + 1]) reads
 * row j = rows[i] of a (rows NULL: j = i), and
 *     y[i, n] = a_scale[j] b_scale[e, n] sum_k a[j, k] b[e, n, k]
 * with the sum exact, in integers, then FP32; out[i, n] = y[i, n], or with
 * swiglu out[i, n] = SiLU(y[i, n]) y[i, N/2 + n], rounded once.
 *   a [Ma, K] int8, pitch a_stride (a multiple of 16 elements), a_scale [Ma];
 *   b [E, N, K] int8 contiguous, b_scale [E, N]; offsets [E + 1] int32
 *   (ascending from 0, moe_dispatch's; NULL with E = 1: all rows), rows [M]
 *   int32 or NULL (moe_dispatch's sorted_token); out [M, N or N/2].
 *   a, b, out 16-byte aligned, ws 256-byte aligned.
 * Rows from offsets[E] on are written as zeros. Offsets are clamped to
 * [0, M]; a row index outside [0, Ma) makes its product row NaN and sets
 * MOE_ERR_DEVICE_INDEX in the workspace's error word; a bounded device wait
 * that runs out makes the outputs that are not stored yet NaN and sets
 * MOE_ERR_TIMEOUT. The call adds to that word and never clears it: have it
 * zeroed before the first call, moe_workspace_status reads and clears it.
 *   The form is chosen from the rows per expert; the environment variable
 * MOE_INT8_FORM, read at each call, overrides it for tests and tuning ("vec":
 * integer dot products; "small", "wide": tensor cores, tiles of up to 32 or
 * 256 rows). The sums are exact in every form, and what follows them (the row's
 * scale, the channel's, SiLU) is the same arithmetic: equal outputs bit for bit. */
moe_status moe_matmul_int8(const moe_int8_config* cfg, const int8_t* a, int64_t a_stride,
                           const float* a_scale, const int8_t* b, const float* b_scale,
                           const int32_t* offsets, const int32_t* rows, void* out, void* ws,
                           size_t ws_bytes, void* stream);

typedef enum moe_norm_kind {
    MOE_NORM_LAYER = 0,  /* (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) */
    MOE_NORM_RMS = 1     /* v / sqrt(mean(v^2) + eps) */
} moe_norm_kind;

typedef enum moe_gate_shape {
    MOE_GATE_NONE = 0,     /* 1 */
    MOE_GATE_CHANNEL = 1,  /* [d] FP32 */
    MOE_GATE_ELEMENT = 2   /* [R, d] of the rows' type, at any pitch */
} moe_gate_shape;

typedef struct moe_block_norm_config {
    int32_t R;      /* rows, >= 0 */
    int32_t d;      /* width, at most 2^24 */
    int32_t dtype;  /* moe_dtype of all [R, d] operands */
    int32_t kind;   /* moe_norm_kind, of both norms */
    int32_t post;   /* 0 or 1: the block's output is normalised */
    int32_t gate;   /* moe_gate_shape */
    float alpha;    /* residual scale */
    float eps;      /* >= 0 */
} moe_block_norm_config;

/* The norms on both sides of a block, fused with its gate and the residual (a layer
 * norm by itself is moe_layer_norm, which is made for it; an RMS norm by itself is
 * this call without y):
 *     z  = post ? Norm(y; post_w, post_b) : y       y: the block's output
 *     x' = alpha x + gate z                         the new residual stream
 *     n  = Norm(x'; w, b)                           the next block's input
 * with Norm(v; w, b) = (v - mu) rstd w + b, statistics and arithmetic in FP32,
 * x' and n rounded once each (n is taken of x' before its rounding).
 *   x, y [R, d]. y NULL: no block in front, x' = x, n = Norm(x); then post and
 *   gate are 0 and out is NULL. Vectors [d] are FP32; post_w, w may be NULL
 *   (1), post_b, b too (0; always with MOE_NORM_RMS). gate NULL exactly with
 *   MOE_GATE_NONE.
 *   out [R, d]: x'. n [R, d] or NULL: no norm follows (w and b NULL).
 *   stats: what the backward takes, or NULL. RMS [2, R] FP32: rstd of y, of
 *   x'; layer [4, R]: mean and rstd of y, mean and rstd of x'. A norm that the
 *   call does not take has mean 0 and rstd 1. */
moe_status moe_block_norm(const moe_block_norm_config* cfg, const void* x, int64_t x_stride, const void* y,
                          int64_t y_stride, const void* gate, int64_t gate_stride, const float* post_w,
                          const float* post_b, const float* w, const float* b, void* out, void* n,
                          float* stats, void* stream);

/* Bytes of workspace moe_block_norm_backward needs where it returns a
 * parameter's gradient (the columns' sums). */
moe_status moe_block_norm_backward_workspace_size(const moe_block_norm_config* cfg, size_t* bytes);

/* Gradients of L = sum(dn n) + sum(dxo x') given the forward's y, gate,
 * vectors and stats and, as x, its x' (y NULL: its x). With h = dn w,
 * xh = (x' - mu) rstd, yh = (y - mu_y) rstd_y ([.]: layer norm alone):
 *     t  = dxo + rstd (h - [mean(h)] - xh mean(h xh)),   dx = alpha t (y NULL: t)
 *     dgate = t z, summed over the rows of a MOE_GATE_CHANNEL
 *     k  = t gate post_w,  dy = rstd_y (k - [mean(k)] - yh mean(k yh))
 *                          (post = 0: t gate)
 *     dpost_w = sum_rows t gate yh, dpost_b = sum_rows t gate,
 *     dw = sum_rows dn xh, db = sum_rows dn
 *   dn or dxo may be NULL, not both; without dn w, dw and db are NULL. dx, dy
 *   and an element's dgate [R, d] contiguous, of dtype; dy NULL exactly where
 *   y is. Vectors' gradients [d] FP32, each may be NULL, overwritten (zeros for
 *   R = 0). An element's dgate may be NULL. ws: 16-byte aligned, needed where a
 *   vector's gradient is asked for. Fixed order of sums: bit-reproducible. */
moe_status moe_block_norm_backward(const moe_block_norm_config* cfg, const void* x, int64_t x_stride,
                                   const void* y, int64_t y_stride, const void* gate, int64_t gate_stride,
                                   const float* post_w, const float* post_b, const float* w,
                                   const float* stats, const void* dn, int64_t dn_stride, const void* dxo,
                                   int64_t dxo_stride, void* dx, void* dy, void* dgate, float* dpost_w,
                                   float* dpost_b, float* dw, float* db, void* ws, size_t ws_bytes,
                                   void* stream);

typedef struct moe_adapter_config {
    int32_t T;          /* rows, >= 0, at most 2^24 */
    int32_t d;          /* input width */
    int32_t N;          /* output width */
    int32_t r;          /* rank (smaller ones padded with zeros), 1..256 */
    int32_t E;          /* adapters, 1..1024 */
    int32_t dtype;      /* moe_dtype of x, a and b */
    int32_t out_dtype;  /* moe_dtype of base and out: dtype or MOE_F32 */
} moe_adapter_config;

/* Bytes of workspace moe_adapter_add needs for cfg (0 for T = 0). */
moe_status moe_adapter_add_workspace_size(const moe_adapter_config* cfg, size_t* bytes);

/* Low-rank adapters of many requests beside a shared projection, whose result
 * is base:
 *     out[t] = base[t] + scale[e] (x[t] a[e]^T) b[e]^T,   e the adapter of row t
 * FP32 sums, both products; out rounded once. With an FP32 output the second
 * product takes the inner values scale x a^T whole; with a 16-bit one it takes 16
 * of their 24 bits (BF16; at most 2^-16 of each is left out, where rounding out
 * takes 2^-8) or 22 (FP16; what lies 2^-39 below the row's largest is zero).
 * Infinities and NaN go as in the formula. Rows are grouped by adapter: those of
 * adapter e are rows[offsets[e]] .. rows[offsets[e + 1] - 1], and rows from
 * position offsets[E] on have none: out[t] = base[t].
 *   x [T, d], a [E, r, d], b [E, N, r] (contiguous); scale [E] FP32 or NULL (1);
 *   offsets [E + 1] int32, ascending from 0, at most T; rows [T] int32, each row
 *   once, or NULL (row i at position i); base, out [T, N] at any pitch, base NULL:
 *   zeros. out may be base (the same pointer and pitch: rows without an adapter are
 *   left as they are), else overlaps no input. moe_dispatch with K = 1 and E + 1
 *   experts, the last for rows without an adapter, gives offsets and rows.
 * ws: 256-byte aligned. Offsets are clamped to [0, T]; a row index outside
 * [0, T) is skipped and sets MOE_ERR_DEVICE_INDEX in the workspace's error word,
 * which the call adds to and never clears (where out is base, positions from
 * offsets[E] on are not looked at); a row that no position names is not
 * written, and what a row named twice holds is not specified. A bounded device
 * wait that runs out makes the outputs that are not stored yet NaN and sets
 * MOE_ERR_TIMEOUT.
 *   Rows on 16 bytes and widths and ranks that are multiples of 8 serve best: others
 * never reach the tensor-core form of many rows. a and b whose rank is padded with
 * zeros to a multiple of 8 give the same result of rows without infinities.
 *   The form is chosen from rows, ranks, adapters and alignment; the environment
 * variable MOE_ADAPTER_FORM, read at each call, overrides it for tests and tuning
 * ("few", "many": rows; "many" only where 16-byte rows, widths and ranks that are
 * multiples of 8 and a rank up to 128 allow it). Forms differ in rounding only. */
moe_status moe_adapter_add(const moe_adapter_config* cfg, const void* x, int64_t x_stride, const void* a,
                           const void* b, const float* scale, const int32_t* offsets, const int32_t* rows,
                           const void* base, int64_t base_stride, void* out, int64_t out_stride, void* ws,
                           size_t ws_bytes, void* stream);

/* Synchronises `stream`, then reads and clears the device-side error word of
 * the workspace: MOE_OK, MOE_ERR_TIMEOUT (a bounded device wait ran out and
 * its kernel stopped early; outputs of that call are invalid) or
 * MOE_ERR_DEVICE_INDEX. moe_forward and moe_dispatch clear the word when
 * they start, so the status covers the calls since the last of those. */
moe_status moe_workspace_status(void* ws, void* stream);

/* Instrumentation. While enabled, each moe_forward records CUDA events
 * around each of its kernel stages selected by stage_mask (bit i = stage i;
 * 0xFFFFFFFF = all) on the caller's stream, for up to max_calls calls.
 * moe_timing_end synchronises those events and returns, per stage, the summed
 * milliseconds over the recorded calls. Stage names via moe_stage_name.
 * Events are created/destroyed by the library. Recording an event between
 * two kernels stops the second from overlapping the first's tail, so time
 * only the stages you need. */
moe_status moe_timing_begin(int32_t max_calls, uint32_t stage_mask);
moe_status moe_timing_end(float* stage_ms, int32_t max_stages, int32_t* n_stages,
                          int32_t* n_calls);
const char* moe_stage_name(int32_t stage);

/* Number of kernels this library has launched in this process. */
uint64_t moe_launch_count(void);

/* Sets the limit of every bounded device-side wait (default 1000 ms). */
moe_status moe_set_wait_timeout_ms(int32_t ms);

/* Self-test of the bounded-wait machinery: launches one kernel that waits on
 * a shared-memory barrier nothing ever completes, with a `ms` millisecond
 * limit, then synchronises. Returns MOE_ERR_TIMEOUT when the wait gave up
 * as designed (and the context stays usable), MOE_OK never. */
moe_status moe_selftest_wait_timeout(int32_t ms, void* ws, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_H */
