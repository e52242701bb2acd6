"""Group-limited routing where float64 scores are equal though the logits are
not: the lowest index ranks first."""
import math

import pytest
import torch

from tests.test_gpu_group_route import A, DT, check, rand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("K,n", [(1, 1), (1, 2), (1, 3), (2, 4), (4, 5), (4, 6), (4, 7), (8, 20), (16, 28)])
def test_infinite_logits_behind_a_saturated_one(A, K, n, score, dt):  # noqa: F811
    """n infinite logits from index 1 (rows 0-7), or scattered (8-15); sigmoid(100) is 1 in float64 as well."""
    r = rand(16, 32, seed=K).to(DT[dt])
    r[:, 0] = 100.0
    r[:8, 1:n + 1] = math.inf
    at = rand(32, seed=n).argsort()[:n]
    r[8:, at] = math.inf
    r[4:8, 31] = 90.0
    for renorm in (False, True):
        got = check(A, r, K, score=score, renorm=renorm)
    if score == "sigmoid":
        assert (got["idx"][:8, 0] == 0).all()
    if K <= 8:
        check(A, r, K, 4, 2, None, score, rank=2)
    check(A, r, K, bias=torch.zeros(32, device="cuda"), score=score)
