"""Group-limited routing where float64 scores are equal though the logits are
not: infinite logits beside saturated ones, groups whose best logits tie exactly
next to others that tie in float64 only. The lowest index ranks first."""
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


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("TG", [1, 2, 3])
@pytest.mark.parametrize("best", [
    [100, math.inf, math.inf, math.inf],  # below an exact tie of the border
    [40, 41, 41, 39], [40, 41, 41, 41],
    [41, 40, 40, 42], [40, 40, 42, 40],   # above it
    [100, 50, math.inf, 60], [100, 50, math.inf, math.inf],
    [0.0, 1e-30, 1e-30, -1e-30], [1e-30, 0.0, 0.0, 2e-30],
    [-0.0, 0.0, 0.0, -0.0],
], ids=str)
def test_groups_that_tie_in_float64_only(A, best, TG, score, dt):  # noqa: F811
    """The best logits of four groups, in every order; sigmoids from 37 on are 1 in
    float64, softmax scores of logits 1e-30 apart are equal."""
    from itertools import permutations
    rows = sorted(set(permutations(best)))
    r = -3.0 - rand(len(rows), 4, 8, seed=TG).abs()
    where = torch.arange(len(rows), device="cuda") % 8
    r[torch.arange(len(rows), device="cuda"), :, where] = torch.tensor(rows, dtype=torch.float32, device="cuda")
    check(A, r.reshape(len(rows), 32).to(DT[dt]), 4, 4, TG, None, score, rank=1)
