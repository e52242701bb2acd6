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
