"""The operators on both sides of a block as a block uses them: the norm before it, an
8-bit projection with the adapters of many requests beside it, the norm behind it with
gate and residual, and the same block's norm gradients. Each step against float64 on the
inputs that the step before left; then the whole run on another stream and captured."""
import pytest
import torch

from tests import block_reference as B
from tests.ops_reference import HALF, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    from mixture_experts_ffn_fp32_gb300 import build
    build.build()
    from mixture_experts_ffn_fp32_gb300 import api
    return api


def weights(A, d, f, E, r, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=g, device="cuda")
    p = {"w0": 1 + 0.1 * rand(d), "w1": 1 + 0.1 * rand(d), "post": 0.5 + 0.1 * rand(d), "gate": 0.3 * rand(d)}
    for name, n, k in (("up", f, d), ("down", d, f)):
        q = A.quantize_rows(rand(n, k) / k ** 0.5)
        p[name], p[name + "_scale"] = q["q"][None], q["scale"][None]
        p[name + "_a"] = (rand(E, r, k) / k ** 0.5).bfloat16()
        p[name + "_b"] = (rand(E, n, r) / r ** 0.5).bfloat16()
    p["scale"] = 0.5 + torch.rand(E, generator=g, device="cuda")
    return p


def project(A, p, name, x, plan, E, **kw):
    q = A.quantize_rows(x, **kw)
    base = A.matmul_int8(q["q"], q["scale"], p[name], p[name + "_scale"], **kw)
    return base, A.adapter_add(base, x, p[name + "_a"], p[name + "_b"], plan["offsets"][:E + 1], plan["sorted_token"],
                               p["scale"], **kw)


def block(A, p, x, plan, E, **kw):
    """x [T, d] BF16 -> everything a step leaves."""
    n0 = A.block_norm(x, weight=p["w0"], **kw)
    up_base, up = project(A, p, "up", n0["n"], plan, E, **kw)
    h = torch.nn.functional.silu(up)
    down_base, down = project(A, p, "down", h, plan, E, **kw)
    out = A.block_norm(x, down, weight=p["w1"], post_weight=p["post"], gate=p["gate"], alpha=0.9, **kw)
    return {"n0": n0["n"], "n0_stats": n0["stats"], "up_base": up_base, "up": up, "h": h, "down_base": down_base,
            "down": down, **{"out_" + k: v for k, v in out.items()}}


def close(got, want):
    val, tol = want
    assert ((got.double() - val).abs() <= tol * 1.001 + 1e-30).all()


@pytest.mark.parametrize("T", [1, 60, 3000])
def test_block(A, T):
    d, f, E, r = 256, 384, 5, 16
    p = weights(A, d, f, E, r)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    ids = torch.randint(E + 1, (T, 1), generator=g, device="cuda").int()
    plan = A.dispatch(A.LayerSpec(T=T, d=d, d_ff=f, E=E + 1, K=1), ids, torch.ones(T, 1, device="cuda"))
    s = block(A, p, x, plan, E)
    n0 = B.block_norm(x, None, None, 1.0, None, None, p["w0"], None, False, False, True, 1e-5)
    close(s["n0"], n0["n"])
    close(s["n0_stats"], n0["stats"])
    for name, src in (("up", s["n0"]), ("down", s["h"])):
        q = A.quantize_rows(src)
        sums = q["q"].double() @ p[name][0].double().T * q["scale"].double()[:, None] * p[name + "_scale"].double()
        assert ((s[name + "_base"].double() - sums).abs() <= (HALF[torch.bfloat16] + 4 * U) * sums.abs()).all()
        close(s[name], B.adapter_add(s[name + "_base"], src, p[name + "_a"], p[name + "_b"], plan["offsets"][:E + 1],
                                     plan["sorted_token"], p["scale"], torch.bfloat16, 2))
    out = B.block_norm(x, s["down"], p["gate"], 0.9, p["post"], None, p["w1"], None, False, True, True, 1e-5)
    for k in out:
        close(s["out_" + k], out[k])
    # the gradients of the norms around the block
    dn, dx = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    got = A.block_norm_backward(s["out_x"], s["out_stats"], s["down"], dn, dx, p["w1"], p["post"], gate=p["gate"], alpha=0.9)
    want = B.block_norm_backward(s["out_x"], s["out_stats"], s["down"], dn, dx, p["gate"], 0.9, p["post"], None, p["w1"],
                                 False, True)
    assert set(got) == set(want)
    for k in want:
        close(got[k], want[k])
    # ... and of the norm before it, the residual's gradient joined
    first = A.block_norm_backward(x, s["n0_stats"], None, got["dy"], got["dx"], p["w0"])
    want = B.block_norm_backward(x, s["n0_stats"], None, got["dy"], got["dx"], None, 1.0, None, None, p["w0"], False, False)
    for k in want:
        close(first[k], want[k])


@pytest.mark.parametrize("T", [60, 3000])
def test_block_elsewhere_and_captured(A, T):
    d, f, E, r = 256, 384, 5, 64
    p = weights(A, d, f, E, r)
    x = torch.randn(T, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    ids = torch.randint(E + 1, (T, 1), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").int()
    plan = A.dispatch(A.LayerSpec(T=T, d=d, d_ff=f, E=E + 1, K=1), ids, torch.ones(T, 1, device="cuda"))
    want = block(A, p, x, plan, E)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block(A, p, x, plan, E)
    torch.cuda.current_stream().wait_stream(side)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(A, p, x, plan, E)
    x.copy_(x.flip(0))
    graph.replay()
    want = block(A, p, x, plan, E)
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
