"""Rows at the ends of FP32 in the norms on both sides of a block, and in the layer norm that shares
their arithmetic."""
import math

import pytest
import torch

from tests.test_gpu_adapter import A, DT  # noqa: F401
from tests import block_reference as B

pytestmark = pytest.mark.gpu


def rand(seed, *s):
    return torch.randn(*s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("d,pad", [(16, 0), (100, 3), (1411, 5), (2048, 0), (8192, 0), (16384, 0), (16392, 0), (20001, 3)])
def test_means_of_infinite_rows(A, d, pad, dt):  # noqa: F811
    """A layer norm's mean of a row with infinities of one sign is that infinity, at every width."""
    x = rand(d, 6, d + pad).to(DT[dt])[:, :d]
    x[0, d // 2], x[1, d - 1], x[2, 0] = math.inf, -math.inf, math.inf
    x[3, 1], x[3, d - 2] = math.inf, -math.inf
    x[4, 3] = math.nan
    want = x.double().mean(1)
    v = rand(1, 6, d).to(DT[dt])
    alone = A.block_norm(x, kind="layer")
    post = A.block_norm(v, x, kind="layer", post_weight=torch.ones(d, device="cuda"))
    before = A.block_norm(x, torch.zeros_like(v), kind="layer", post=False)
    for got, at in ((alone, 2), (post, 0), (before, 2)):
        mean, rstd = got["stats"][at], got["stats"][at + 1]
        assert torch.equal(mean[:3], want[:3].float()) and mean[3:5].isnan().all()
        assert rstd[:5].isnan().all() and got["n"][:5].isnan().all() and got["n"][5].isfinite().all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [10, 24, 37, 40, 56, 72, 100, 120])
def test_constant_rows_of_large_values(A, d, dt):  # noqa: F811
    """Constant rows whose mean times 1 / deviation passes FP32's range: x - mean is zero in the row, and what
    lies behind its end counts as nothing."""
    R = 9
    value = torch.where(torch.arange(R, device="cuda") % 3 == 0, 1.0, 2.0 ** 120).to(DT[dt])
    const = value[:, None].expand(R, d).contiguous()
    vec = [1 + 0.1 * rand(i, d) for i in range(3)] + [0.1 * rand(3, d)]
    dn, dx = rand(4, R, d).to(DT[dt]), rand(5, R, d).to(DT[dt])

    def check(got, want):
        for k, (v, tol) in want.items():
            assert ((got[k].double() - v).abs() <= tol * 1.001 + 1e-30).all(), k

    mean, rstd = value.float(), torch.full((R,), 1e-5 ** -0.5, device="cuda")
    first = torch.stack([0 * mean, 0 * mean + 1, mean, rstd])
    check(A.block_norm_backward(const, first, dn=dn, weight=vec[0], kind="layer"),
          B.block_norm_backward(const, first, None, dn, None, None, 1.0, None, None, vec[0], True, False))
    st = torch.stack([mean, rstd, mean, rstd])
    for gate in (None, vec[2], torch.sigmoid(rand(6, R, d)).to(DT[dt])):
        check(A.block_norm_backward(const, st, y=const, dn=dn, dx=dx, weight=vec[0], post_weight=vec[1], post_bias=vec[3],
                                    gate=gate, alpha=0.5, kind="layer"),
              B.block_norm_backward(const, st, const, dn, dx, gate, 0.5, vec[1], vec[3], vec[0], True, True))
    got = A.layer_norm_backward(dn, const, mean, rstd, vec[0])
    want = B.block_norm_backward(const, first, None, dn, None, None, 1.0, None, None, vec[0], True, False)
    check({"dx": got["dx"], "dweight": got["dweight"], "dbias": got["dbias"]}, want)
