"""A pre-norm MoE block from the operators around the layer.

Serving: layer norm, group-limited routing, dispatch, then the experts in 8 bits
(row quantisation, gate/up product with the SwiGLU epilogue, quantisation, down
product), and the weighted sum per token added to the residual:

    x + sum_k w_k Expert_{e_k}(LN(x))

Training: the gradient that the router's weights take back through the routing
and the norm. Run as a program it builds a small random block, does both and
prints how far the 8-bit block is from the same block in FP32.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_ffn_fp32_gb300 import api  # noqa: E402

GROUPS = dict(n_groups=4, topk_groups=2, score="sigmoid", group_rank=2, renormalize=True, scale=1.0)


def make_block(d, d_ff, E, seed=0, device="cuda"):
    """Random weights of a block, the experts' also as the 8-bit product takes them."""
    g = torch.Generator(device=device).manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=g, device=device)

    p = {"gamma": 1 + 0.1 * rand(d), "beta": 0.1 * rand(d), "W_router": rand(d, E) / d ** 0.5,
         "bias": 0.01 * rand(E), "gate_up": rand(E, d, 2 * d_ff) / d ** 0.5, "down": rand(E, d_ff, d) / d_ff ** 0.5}
    for name in ("gate_up", "down"):
        w = p[name].transpose(1, 2)  # [E, channels, reduction]
        q = api.quantize_rows(w.reshape(-1, w.shape[2]))
        p[name + "_q"], p[name + "_scale"] = q["q"].view(w.shape), q["scale"].view(w.shape[:2])
    return p


def serve(p, x, K):
    """The block's forward on tokens x [T, d] (BF16), the experts in 8 bits."""
    T, d = x.shape
    E = p["W_router"].shape[1]
    n = api.layer_norm(x, p["gamma"], p["beta"])["y"]
    r = api.group_route(n.float() @ p["W_router"], K, bias=p["bias"], **GROUPS)
    spec = api.LayerSpec(T=T, d=d, d_ff=p["down"].shape[1], E=E, K=K)
    dp = api.dispatch(spec, r["idx"], r["w"])
    a = api.quantize_rows(n)
    h = api.matmul_int8(a["q"], a["scale"], p["gate_up_q"], p["gate_up_scale"], offsets=dp["offsets"],
                        rows=dp["sorted_token"], swiglu=True)
    b = api.quantize_rows(h)
    # the routing weights ride on the rows' scales
    y = api.matmul_int8(b["q"], b["scale"] * dp["sorted_w"], p["down_q"], p["down_scale"], offsets=dp["offsets"],
                        out_dtype="f32")
    there = r["idx"] >= 0  # slots that routing left empty hold no row
    rows = torch.where(there, dp["inv"], 0).long()
    return (x.float() + (y[rows.view(-1)].view(T, K, d) * there[:, :, None]).sum(1)).to(x.dtype), r


def reference(p, x, r):
    """The same block in FP32 on the routing r."""
    xf = x.float()
    n = torch.nn.functional.layer_norm(xf, xf.shape[1:], p["gamma"], p["beta"])
    out = xf.clone()
    for e in range(p["W_router"].shape[1]):
        t, k = (r["idx"] == e).nonzero(as_tuple=True)
        a, u = (n[t] @ p["gate_up"][e]).chunk(2, 1)
        out.index_add_(0, t, r["w"][t, k, None] * ((torch.nn.functional.silu(a) * u) @ p["down"][e]))
    return out


def router_gradients(p, x, K, dw):
    """Gradients of sum(dw * w) with respect to W_router, gamma, beta and x, the
    selection held fixed."""
    f = api.layer_norm(x, p["gamma"], p["beta"])
    logits = f["y"].float() @ p["W_router"]
    r = api.group_route(logits, K, bias=p["bias"], **GROUPS)
    dl = api.group_route_backward(dw, r["idx"], logits, score=GROUPS["score"], renormalize=GROUPS["renormalize"],
                                  scale=GROUPS["scale"])
    dn = (dl @ p["W_router"].T).to(x.dtype)
    b = api.layer_norm_backward(dn, x, f["mean"], f["rstd"], p["gamma"])
    return {"dW_router": f["y"].float().T @ dl, "dgamma": b["dweight"], "dbeta": b["dbias"], "dx": b["dx"]}, r


def main():
    T, d, d_ff, E, K = 512, 256, 128, 32, 4
    p = make_block(d, d_ff, E)
    x = torch.randn(T, d, device="cuda").bfloat16()
    out, r = serve(p, x, K)
    ref = reference(p, x, r)
    err = (out.float() - ref).norm() / (ref - x.float()).norm()
    print(f"8-bit block against FP32: relative error of the experts' part {float(err):.4f}")
    grads, _ = router_gradients(p, x, K, torch.randn(T, K, device="cuda"))
    for name, g in grads.items():
        print(f"{name} {tuple(g.shape)}: norm {float(g.float().norm()):.4f}")


if __name__ == "__main__":
    main()
