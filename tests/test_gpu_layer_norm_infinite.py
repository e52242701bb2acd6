"""Layer norm of rows with infinities: the mean is the sum's, the rest of the row no number."""
import math

import pytest
import torch

from tests.test_gpu_layer_norm import A, DT, rand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("d,pad", [(16, 0), (26, 0), (100, 3), (384, 0), (640, 0), (1411, 5), (2048, 0), (5120, 0),
                                   (8192, 0), (16384, 0), (16392, 0)])
def test_rows_with_infinities(A, d, pad, dt):  # noqa: F811
    x = rand((6, d), d, 1.0, DT[dt], pad)
    x[0, d // 2] = math.inf
    x[1, d - 1] = -math.inf
    x[2, 0], x[2, d - 1] = math.inf, math.inf
    x[3, 1], x[3, d - 2] = math.inf, -math.inf
    x[4, 3] = math.nan
    got = A.layer_norm(x)
    want = x.double().mean(1)
    assert torch.equal(got["mean"][:3], want[:3].float()) and got["mean"][3:5].isnan().all()
    assert got["rstd"][:5].isnan().all() and got["y"][:5].isnan().all()
    alone = A.layer_norm(x[5:])
    assert all(torch.equal(got[k][5:], alone[k]) for k in got) and got["y"][5].isfinite().all()
