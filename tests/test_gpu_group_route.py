"""Group-limited routing against float64: the selection equal, the weights and
gradients within counted roundings; masked experts, empty rows, ties, scores
next to each other, odd group sizes."""
import math

import pytest
import torch

from tests import ops_reference as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def A():
    from mixture_experts_ffn_fp32_gb300 import build
    build.build()
    from mixture_experts_ffn_fp32_gb300 import api
    return api


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def check(A, r, K, G=1, TG=1, bias=None, score="sigmoid", rank=2, renorm=True, scale=1.0):
    got = A.group_route(r, K, n_groups=G, topk_groups=TG, bias=bias, score=score, group_rank=rank,
                        renormalize=renorm, scale=scale)
    idx, w = R.group_route(r, K, G, TG, bias, score, rank, renorm, scale)
    assert torch.equal(got["idx"].cpu(), idx)
    # exponential and division 4 U, sums of E terms in chains of 8 and a tree of 5, argument 2 U
    tol = 32 * R.U * w.abs() + 1e-37
    assert ((got["w"].cpu().double() - w).abs() <= tol).all()
    return got


# T, E, K, G, TG: one token, one expert, groups across lanes, groups of 5, 20, 45 and 3 experts
SHAPES = [(1, 1, 1, 1, 1), (5, 8, 2, 2, 1), (130, 32, 4, 4, 2), (77, 64, 6, 8, 3), (33, 96, 5, 6, 2),
          (200, 128, 8, 8, 4), (64, 160, 8, 8, 3), (65, 160, 3, 32, 7), (100, 225, 7, 5, 2), (257, 256, 8, 8, 4),
          (40, 256, 16, 32, 9), (50, 256, 8, 1, 1), (30, 9, 3, 3, 1), (20, 254, 5, 2, 1), (16, 17, 16, 1, 1),
          (12, 256, 16, 2, 2)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_route(A, shape, score, dt):
    T, E, K, G, TG = shape
    r = rand(T, E, seed=T).to(DT[dt])
    b = 0.1 * rand(E, seed=E)
    for bias in (None, b):
        for rank in (1, 2):
            check(A, r, K, G, TG, bias, score, rank, renorm=rank == 2, scale=2.5 if rank == 1 else 1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masked_experts(A, score):
    """-inf and NaN logits, -inf and NaN biases: never taken; rows with fewer
    eligible experts than slots end in -1; empty rows are all -1, weight 0."""
    r = rand(64, 64, seed=3)
    r[0] = -math.inf
    r[1] = math.nan
    r[2, 3:] = -math.inf
    r[3, ::2] = math.nan
    r[4:20, 8:48] = -math.inf
    r[20] = torch.finfo(torch.float32).min
    r[21, :60] = torch.finfo(torch.float32).min
    bias = 0.05 * rand(64, seed=4)
    bias[5], bias[9] = -math.inf, math.nan
    for b in (None, bias):
        for G, TG in ((1, 1), (8, 2), (4, 3)):
            got = check(A, r, 6, G, TG, b, score)
            assert (got["idx"][0] == -1).all() and (got["w"][:2] == 0).all()
            assert (got["idx"][2] >= 0).sum() == 3
            if b is not None:
                assert not ((got["idx"] == 5) | (got["idx"] == 9)).any()


def test_all_ties_take_the_lowest(A):
    r = torch.zeros(9, 128, device="cuda")
    for score in ("sigmoid", "softmax"):
        got = check(A, r, 8, 8, 2, None, score)
        assert torch.equal(got["idx"].cpu(), torch.arange(8, dtype=torch.int32).expand(9, 8))
        check(A, r, 8, 8, 2, torch.full((128,), -0.25, device="cuda"), score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
def test_next_to_each_other(A, score, biased):
    """Logits a few units in the last place apart: FP32 scores cannot order them."""
    T, E = 400, 64
    base = 1.0 + 0.5 * rand(T, 1, seed=5)
    step = torch.randint(-4, 5, (T, E), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    r = base * (1 + step * 2.0 ** -23)
    bias = None
    if biased:
        bias = 0.25 + torch.randint(-3, 4, (E,), generator=torch.Generator(device="cuda").manual_seed(7),
                                    device="cuda") * 2.0 ** -26
    check(A, r, 8, 1, 1, bias, score)
    check(A, r, 8, 8, 3, bias, score, rank=1)
    check(A, r, 8, 8, 3, bias, score, rank=2)


def test_saturated_and_tiny_scores(A):
    r = rand(128, 32, seed=8) * 60
    for score in ("sigmoid", "softmax"):
        for renorm in (False, True):
            check(A, r, 6, 4, 2, None, score, renorm=renorm)
    low = -150 + rand(32, 32, seed=9)  # sigmoids below FP32's range still share the weight
    got = check(A, low, 4, renorm=True)
    assert ((got["w"].sum(1) - 1).abs() < 1e-6).all()
    inf = rand(8, 32, seed=10)
    inf[:, 3] = math.inf
    inf[2:, 17] = math.inf
    check(A, inf, 2, score="softmax", renorm=True)
    check(A, inf, 2, score="sigmoid", renorm=False)


def test_large_bias(A):
    r = rand(200, 64, seed=11)
    bias = 1000.0 + rand(64, seed=12)
    bias[::3] *= -1
    check(A, r, 8, 8, 4, bias, "sigmoid")
    check(A, r, 8, 8, 4, bias, "softmax")


def test_strided_rows_streams_graph(A):
    wide = rand(100, 259, seed=13)
    r = wide[:, 1:257]
    got = check(A, r, 8, 8, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = A.group_route(r, 8, n_groups=8, topk_groups=4, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other["idx"], got["idx"]) and torch.equal(other["w"], got["w"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = A.group_route(r, 8, n_groups=8, topk_groups=4)
        d = A.group_route_backward(g["w"], g["idx"], r)
    wide.copy_(rand(100, 259, seed=14))
    graph.replay()
    want = check(A, r, 8, 8, 4)
    assert torch.equal(g["idx"], want["idx"])
    assert torch.equal(d, A.group_route_backward(want["w"], want["idx"], r))
    assert A.group_route(r[:0], 8)["idx"].shape == (0, 8)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(A, shape, score, renorm, dt):
    T, E, K, G, TG = shape
    r = rand(T, E, seed=T + 1).to(DT[dt])
    if T > 4 and E > K:
        r[0] = -math.inf
        r[1, K - 1:] = -math.inf
    f = A.group_route(r, K, n_groups=G, topk_groups=TG, score=score, renormalize=renorm, scale=1.5)
    dw = rand(T, K, seed=T + 2)
    got = A.group_route_backward(dw, f["idx"], r, score=score, renormalize=renorm, scale=1.5)
    assert got.dtype == r.dtype
    rd = r.double().clone()
    empty = (rd == -math.inf).all(1)
    rd[empty] = 0.0  # no selection there: no gradient
    rd.requires_grad_(True)
    w = R.group_weights(rd, f["idx"], score, renorm, 1.5)
    (w * dw.double()).sum().backward()
    want = rd.grad
    want = torch.where(want.isnan(), 0.0, want)
    # terms of the difference at most 1.5 max|dw|, times the score they weigh: 48 U of that
    s = R.scores(r, score)
    idx = f["idx"].long()
    sel = torch.where(idx >= 0, s.gather(1, idx.clamp(min=0)), 0.0)
    weigh = sel / sel.sum(1, keepdim=True).clamp(min=1e-300) if renorm else sel
    big = 1.5 * dw.double().abs().max(1, keepdim=True).values
    mag = torch.zeros_like(s).scatter_add_(1, idx.clamp(min=0), weigh)
    if score == "softmax" and not renorm:
        mag = mag + s * sel.sum(1, keepdim=True)
    tol = 48 * R.U * big * mag * K ** 0.5 + R.HALF[r.dtype] * want.abs() + (6e-8 if dt == "f16" else 1e-37)
    assert ((got.double() - want).abs() <= tol).all()
    if T > 4 and E > K:
        assert (got[0] == 0).all()


def test_backward_against_differences(A):
    r = rand(3, 12, seed=20)
    dw = rand(3, 4, seed=21)
    for score in ("sigmoid", "softmax"):
        for renorm in (False, True):
            f = A.group_route(r, 4, n_groups=3, topk_groups=2, score=score, renormalize=renorm)
            got = A.group_route_backward(dw, f["idx"], r, score=score, renormalize=renorm)
            rd = r.double()
            for i in range(3):
                for e in range(12):
                    d = torch.zeros_like(rd)
                    d[i, e] = 1e-6
                    hi = (R.group_weights(rd + d, f["idx"], score, renorm, 1.0) * dw.double()).sum()
                    lo = (R.group_weights(rd - d, f["idx"], score, renorm, 1.0) * dw.double()).sum()
                    assert abs(float(hi - lo) / 2e-6 - float(got[i, e])) < 2e-6


def test_backward_skips_foreign_ids(A):
    r = rand(4, 16, seed=22)
    idx = torch.tensor([[0, 99], [-1, -7], [3, 16], [15, 2]], dtype=torch.int32, device="cuda")
    dw = torch.ones(4, 2, device="cuda")
    got = A.group_route_backward(dw, idx, r, renormalize=False)
    s = torch.sigmoid(r.double())
    want = torch.zeros_like(s)
    for i, e in ((0, 0), (2, 3), (3, 15), (3, 2)):
        want[i, e] = s[i, e] * (1 - s[i, e])
    assert ((got.double() - want).abs() <= 1e-6).all()


def test_logits_that_float64_scores_cannot_tell_apart(A):
    """Sigmoids that round to the same float64 (logits above 20), scores below its
    range, and logits within 1e-12: equal there, so the lowest index is taken."""
    E = 32
    base = torch.tensor([0.0, 5.0, 15.0, 21.0, 25.0, 33.0, 40.0, 85.0, -30.0, -600.0, -720.0, -1000.0], device="cuda")
    r = base[:, None].repeat(1, E)
    up = torch.arange(E, device="cuda") % 5
    for _ in range(4):
        r = torch.where(up[None] > 0, torch.nextafter(r, torch.full_like(r, 1e4)), r)
        up = up - 1
    tiny = torch.zeros(2, E, device="cuda")
    tiny[0, 7], tiny[1, 9] = 1e-30, 1e-9
    r = torch.cat([r, tiny])
    top = r.clone()
    top[:, 3] = 90.0  # softmax maximum far above the others
    for score in ("sigmoid", "softmax"):
        for x in (r, top):
            check(A, x, 6, 1, 1, None, score)
            check(A, x, 6, 4, 2, None, score, rank=1)
            check(A, x, 6, 4, 2, None, score, rank=2)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_zeros_of_both_signs_are_equal(A, score, dt):
    sign = torch.where(rand(64, 256, seed=7) > 0, 1.0, -1.0)
    r = (0.0 * sign).to(DT[dt])
    r[:, 200] = -1.0
    for G, TG, rank in [(1, 1, 2), (8, 3, 1), (8, 3, 2)]:
        got = check(A, r, 8, G, TG, None, score, rank)
        assert torch.equal(got["idx"].cpu(), torch.arange(8, dtype=torch.int32).expand(64, 8))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("step", [0.5, 2.0 ** -7, 2.0 ** -24])
def test_ties_of_coarse_logits(A, score, dt, step):
    """Runs of equal logits across the last rank, next to others a step away."""
    r = (torch.round(2.0 * rand(300, 96, seed=11)) * step).to(DT[dt])
    r[150:] += torch.tensor(1.5, dtype=DT[dt], device="cuda")
    for G, TG, rank in [(1, 1, 2), (6, 2, 1), (6, 2, 2)]:
        check(A, r, 5, G, TG, None, score, rank)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("at", [(3, 5), (3, 20), (3, 5, 6), (0, 8, 31)], ids=str)
def test_group_sums_next_to_each_other(A, score, biased, at):
    """Groups whose two best sum to nearly the same, wherever in the group they
    are, with a third best next to the second."""
    T, G, n = 200, 8, 32
    r = -3.0 + 0.5 * rand(T, G, n, seed=21)
    ulps = torch.randint(-3, 4, (T, G, len(at)), generator=torch.Generator(device="cuda").manual_seed(22),
                         device="cuda")
    best = 2.0 + 0.5 * rand(T, 1, 1, seed=23) - torch.tensor([0.0, 0.25, 0.25], device="cuda")[:len(at)]
    r[:, :, list(at)] = best * (1 + ulps * 2.0 ** -23)
    bias = 0.1 * rand(1, n, seed=24).expand(G, n).reshape(-1).contiguous() if biased else None
    check(A, r.reshape(T, G * n), 8, G, 3, bias, score, rank=2)
