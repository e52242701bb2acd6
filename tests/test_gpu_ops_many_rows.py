"""The operators around the layer past the first turn of their loops: more rows
than the resident CTAs take at a time, so that rings wrap, tiles follow tiles in a
CTA pair and tokens that need FP64 come in later turns."""
import math

import pytest
import torch

from tests import ops_reference as R
from tests import test_gpu_group_route as route
from tests import test_gpu_int8 as int8
from tests import test_gpu_layer_norm as norm
from tests.test_gpu_int8 import A, DT, gen, ints, rand  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- 8-bit products: 13 row tiles of 256 (or 84 of 32) by 16 or 32 channel tiles ----

@pytest.mark.parametrize("form", ["wide", "small"])
@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("chunks", [1, 2])
def test_tiles_after_tiles(A, monkeypatch, form, out, swiglu, chunks):  # noqa: F811
    """chunks 2: rows whose sum of |a| passes 2^17, so that integers are summed from two accumulators."""
    monkeypatch.setenv("MOE_INT8_FORM", form)
    M, E, N, K = 2700, 3, 4096, 272 if chunks == 1 else 1296
    a, b = ints(M, K, seed=1), ints(E, N, K, seed=2)
    if chunks == 2:
        a = torch.where(a < 0, a.clamp(max=-112), a.clamp(min=112))
        assert int(a.int().abs().sum(1).max()) > 2 ** 17
    sa = 0.5 + torch.rand(M, generator=gen(3), device="cuda")
    sb = (0.5 + torch.rand(E, N, generator=gen(4), device="cuda")) / (5000 * K ** 0.5)
    int8.check(A, a, sa, b, sb, [0, 1100, 1100, 2690], None, swiglu, out)


# ---- 8-bit products: the border between one accumulator and chunks ----

@pytest.mark.parametrize("form", ["vec", "small", "wide"])
@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("past", [False, True])
def test_one_accumulator_at_its_limit(A, monkeypatch, form, M, past):  # noqa: F811
    """Rows whose |a| sums to 2^17 exactly, and to 3 more: all products of one sign, up to
    2^24, the last ones odd (an FP32 sum past 2^24 would lose them)."""
    monkeypatch.setenv("MOE_INT8_FORM", form)
    K, N = 1200, 70
    a = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    b = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
    b[0, ::3] = -127
    if past:
        a[:, :1024] = -128
        for k in (1100, 1140, 1199):
            a[:, k] = 1
            b[0, :, k] = 1
        a[1::2, 1100] = 0
    else:
        a[:, :1023] = -128
        a[:, 1100], a[:, 1199] = -127, -1
        b[0, 1::2, 1199] = -1
    assert int(a.int().abs().sum(1).max()) == 2 ** 17 + (3 if past else 0)
    got = A.matmul_int8(a, torch.ones(M, device="cuda"), b, torch.ones(1, N, device="cuda"), out_dtype="f32")
    want = (a.cpu().double() @ b[0].cpu().double().T).float()
    assert torch.equal(got.cpu(), want)


# ---- 8-bit products: every check of rows, scales and streams in every form ----

@pytest.fixture(params=["vec", "small", "wide"])
def form(request, monkeypatch):
    monkeypatch.setenv("MOE_INT8_FORM", request.param)
    return request.param


@pytest.mark.parametrize("M", [6, 700])
@pytest.mark.parametrize("av,bv", [(127, 127), (-128, -128), (-128, 127), (101, 127)])
def test_extreme_sums(A, form, M, av, bv):  # noqa: F811
    int8.test_extreme_sums_are_exact(A, M, av, bv)


@pytest.mark.parametrize("M", [5, 900])
def test_rows(A, form, M):  # noqa: F811
    int8.test_rows_without_an_expert_are_zero(A, M)
    int8.test_bad_row_index_is_reported(A, max(M, 6))
    int8.test_bad_offsets_stay_in_bounds(A, M)
    int8.test_nan_scales_reach_the_output(A)


@pytest.mark.parametrize("M", [0, 4, 700])
def test_streams_and_graphs(A, form, M):  # noqa: F811
    int8.test_stream_graph_and_workspace(A, M)


@pytest.mark.parametrize("shape", [(64, 7, 8, 192, 80), (700, 2000, 4, 1088, 264)], ids=str)
def test_gathered(A, form, shape):  # noqa: F811
    int8.test_gathered_rows(A, shape)


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("shape", [(257, 1, 1040, 130), (1000, 4, 512, 256), (513, 64, 320, 72)], ids=str)
def test_every_output(A, form, shape, swiglu, out):  # noqa: F811
    int8.test_matmul(A, shape, swiglu, out)


# ---- rows to 8 bits: at least three turns of each width's CTAs ----

@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", [(60007, 16, 0), (60001, 96, 0), (16003, 300, 0), (15001, 512, 8), (12001, 1024, 0),
                                   (5003, 1280, 0), (4003, 2048, 0), (4001, 2048, 1), (2903, 2560, 0), (2001, 4096, 0),
                                   (1303, 6144, 0), (1003, 8192, 0), (503, 16384, 0)], ids=str)
def test_quantize(A, shape, dt):  # noqa: F811
    int8.test_quantize_rows(A, shape, dt)


# ---- layer norm ----

@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", [(70001, 16, 0), (50003, 64, 0), (40001, 100, 0), (33001, 128, 0), (20003, 320, 0),
                                   (16001, 512, 3), (9001, 1024, 0), (4001, 1536, 0), (4003, 2048, 0), (3001, 2048, 1),
                                   (2003, 4096, 0), (1001, 8192, 0), (701, 16384, 0)], ids=str)
def test_norm(A, shape, dt):  # noqa: F811
    norm.test_forward(A, shape, dt)
    if shape[1] <= 8192:
        norm.test_backward(A, shape, dt)


# ---- routing: a turn holds 19456 tokens, the outer loop's step 32 of them ----

def logits_with_near_ones(T, E, dt, seed):
    """Every 97th token's logits are a few steps of FP32 apart, every 101st's equal in pairs."""
    r = rand(T, E, seed=seed)
    step = torch.randint(-4, 5, (T, E), generator=gen(seed + 1), device="cuda")
    r[::97] = (r[::97, :1] * (1 + step[::97] * 2.0 ** -23))
    r[::101, 1::2] = r[::101, ::2]
    r[::307] = -math.inf
    return r.to(dt)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("E,G,TG,biased", [(32, 4, 2, False), (32, 1, 1, True), (96, 6, 2, True)])
def test_route(A, E, G, TG, biased, dt, score):  # noqa: F811
    r = logits_with_near_ones(40007, E, DT[dt], E)
    bias = 0.25 + torch.randint(-3, 4, (E,), generator=gen(7), device="cuda") * 2.0 ** -26 if biased else None
    route.check(A, r, 4, G, TG, bias, score, rank=2 if biased else 1)


@pytest.mark.parametrize("biased", [False, True])
def test_route_256(A, biased):  # noqa: F811
    bias = 0.1 * rand(256, seed=9) if biased else None
    route.check(A, logits_with_near_ones(19999, 256, torch.float32, 8), 8, 8, 4, bias, "sigmoid")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dt", list(DT))
def test_route_past_the_outer_loop(A, dt, score):  # noqa: F811
    T, E, K = 640003, 8, 2
    r = logits_with_near_ones(T, E, DT[dt], 3)
    got = A.group_route(r, K, score=score)
    s = R.scores(r, score)
    val, idx = torch.where(r > -math.inf, s, -math.inf).sort(dim=1, descending=True, stable=True)
    val, idx = val[:, :K], idx[:, :K]
    none = val == -math.inf
    assert torch.equal(got["idx"].long(), torch.where(none, -1, idx))
    sel = torch.where(none, 0.0, val)
    w = sel / sel.sum(1, keepdim=True).clamp(min=1e-300)
    assert ((got["w"].double() - w).abs() <= 32 * R.U * w + 1e-37).all()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shape", [(30011, 32, 4, 4, 2), (20003, 160, 8, 8, 3)], ids=str)
def test_route_backward(A, shape, score, renorm, dt):  # noqa: F811
    route.test_backward(A, shape, score, renorm, dt)
