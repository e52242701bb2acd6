"""The example block: the operators together, as they would be used."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_ffn_fp32_gb300 import build
    build.build()
    from examples import moe_block
    return moe_block


@pytest.mark.parametrize("T", [1, 7, 200, 3000])
def test_serve(B, T):
    """A value quantised by its row's maximum is off by a step's 1 / sqrt(12) of
    max / 127: 0.9 % of the row's deviation where the maximum is 4 of them. Four
    such roundings (two operands of two products) and BF16's of the output
    stay within 4 %."""
    p = B.make_block(256, 128, 32)
    x = torch.randn(T, 256, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").bfloat16()
    out, r = B.serve(p, x, 4)
    ref = B.reference(p, x, r)
    assert (r["idx"] >= 0).all()
    assert float((out.float() - ref).norm() / (ref - x.float()).norm()) < 0.04


def test_router_gradients(B):
    p = B.make_block(128, 64, 32)
    x = torch.randn(300, 128, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    dw = torch.randn(300, 4, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    got, r = B.router_gradients(p, x, 4, dw)
    leaves = {k: p[k].double().requires_grad_(True) for k in ("W_router", "gamma", "beta")}
    leaves["x"] = x.double().requires_grad_(True)
    n = torch.nn.functional.layer_norm(leaves["x"], (128,), leaves["gamma"], leaves["beta"])
    s = (n @ leaves["W_router"]).sigmoid().gather(1, r["idx"].long())
    (dw.double() * s / s.sum(1, keepdim=True)).sum().backward()
    for name, leaf in leaves.items():
        want = leaf.grad
        # FP32 through two products of 128 and 300 terms
        assert float((got["d" + name].double() - want).norm() / want.norm()) < 2e-5, name
