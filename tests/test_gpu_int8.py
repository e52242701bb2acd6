"""Row quantisation and the 8-bit expert products against float64: q equal,
sums exact, outputs within counted roundings; ragged experts, gathered rows,
odd channel counts, extreme sums, rows that no expert covers."""
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=gen(seed), device="cuda")


def ints(*shape, seed=0, lo=-128, hi=128):
    return torch.randint(lo, hi, shape, generator=gen(seed), device="cuda", dtype=torch.int32).to(torch.int8)


# ---- quantisation ----

@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", [(1, 1, 0), (3, 16, 0), (70, 96, 0), (33, 250, 3), (64, 1000, 0), (9, 1411, 5),
                                   (40, 2048, 0), (17, 4096, 8), (3, 8200, 0), (2, 20000, 1), (5001, 64, 0), (333, 128, 8),
                                   (700, 100, 3), (9, 8192, 0)], ids=str)
def test_quantize_rows(A, shape, dt):
    n, k, pad = shape
    x = (rand(n, k + pad, seed=k) * 3).to(DT[dt])[:, :k]
    got = A.quantize_rows(x)
    q, scale = R.quantize_rows(x)
    assert torch.equal(got["scale"], scale) and torch.equal(got["q"], q)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", [(900, 1280, 0), (700, 1536, 3), (600, 2560, 8), (31, 2561, 0), (400, 5120, 0),
                                   (65, 6144, 1)], ids=str)
def test_quantize_three_quarter_widths(A, shape, dt):
    test_quantize_rows(A, shape, dt)


@pytest.mark.parametrize("dt", list(DT))
def test_quantize_coarse_values(A, dt):
    """Few significant bits: quotients on half steps, and next to them by the
    scale's own rounding, in every row."""
    x = torch.randint(-64, 65, (300, 1000), generator=gen(40), device="cuda").float() * \
        2.0 ** torch.randint(-20, 20, (300, 1), generator=gen(41), device="cuda")
    x[:, 0] = x.abs().amax(1) * (1 + torch.arange(300, device="cuda") % 4 * 0.25)
    x = x.to(DT[dt])
    got = A.quantize_rows(x)
    q, scale = R.quantize_rows(x)
    assert torch.equal(got["scale"].nan_to_num(-1), scale.nan_to_num(-1)) and torch.equal(got["q"], q)


def test_quantize_half_steps(A):
    """Quotients on and next to half steps: x = scale (n + 1/2) exactly, and one unit off."""
    n = torch.arange(-127, 127, device="cuda", dtype=torch.float32) + 0.5
    rows = []
    for scale in (1.0, 2.0 ** -7, 0.75, 3.0 * 2.0 ** -20, 1 / 3, 0.1):
        s = torch.tensor(scale, device="cuda")
        h = n * s
        rows.append(torch.cat([h, torch.nextafter(h, h + 1), torch.nextafter(h, h - 1), s[None] * 127, -s[None] * 127]))
    x = torch.stack(rows)
    got = A.quantize_rows(x)
    q, scale = R.quantize_rows(x)
    assert torch.equal(got["scale"], scale) and torch.equal(got["q"], q)


def test_quantize_extremes(A):
    x = rand(10, 64, seed=1)
    x[0] = 0
    x[1, 3] = math.inf
    x[2, 5] = math.nan
    x[3] *= 1e-38
    x[4] *= 1e-43
    x[5] = 3e38 * torch.sign(x[5])
    x[6] = 1e-45
    x[7, 0] = 1e30
    got = A.quantize_rows(x)
    q, scale = R.quantize_rows(x)
    assert torch.equal(got["q"], q) and torch.equal(got["scale"].nan_to_num(-1), scale.nan_to_num(-1))
    assert (got["q"][:3] == 0).all() and got["scale"][0] == 0 and got["scale"][1:3].isnan().all()
    assert A.quantize_rows(x[:0])["q"].shape == (0, 64)


# ---- products ----

def splits_of(E, M, seed):
    """Ascending offsets with empty experts among them."""
    g = torch.Generator().manual_seed(seed)
    if E == 1:
        return [0, M]
    cut = torch.randint(0, M + 1, (E - 1,), generator=g).sort().values.tolist()
    if E > 3:
        cut[0] = 0
        cut[-1] = M
    return [0] + cut + [M]


def check(A, a, sa, b, sb, splits=None, rows=None, swiglu=False, out="f32", ws=None):
    E, N, K = b.shape
    M = a.shape[0] if rows is None else rows.shape[0]
    offsets = None if splits is None else torch.tensor(splits, dtype=torch.int32, device="cuda")
    got = A.matmul_int8(a, sa, b, sb, offsets=offsets, rows=rows, swiglu=swiglu, out_dtype=out, ws=ws)
    sp = [0, M] if splits is None else splits
    want, gate = R.matmul_int8(a, sa, b, sb, sp, rows, swiglu)
    g = got[:sp[-1]].cpu().double()
    assert got.shape == (M, N // 2 if swiglu else N) and (got[sp[-1]:] == 0).all()
    # the integer sum to FP32, two scales: 3 roundings; SiLU: its argument's, an
    # exponential of 2 units, a sum, a division and two products
    rel = 4 * R.U if gate is None else R.U * (16 + 4 * gate)
    tol = rel * want.abs() + R.HALF[got.dtype] * want.abs() * 1.001 + (6e-8 if out == "f16" else 1e-37)
    assert ((g - want).abs() <= tol).all(), float(((g - want).abs() - tol).max())
    return got


# M, E, K, N: single rows, one channel, few rows per expert, tiles and their
# edges, reductions past one exact chunk, odd channel counts
SHAPES = [(1, 1, 16, 1), (1, 1, 4096, 64), (3, 1, 48, 37), (9, 4, 64, 96), (40, 8, 256, 130), (16, 256, 128, 64),
          (130, 1, 1024, 128), (257, 1, 1040, 129), (300, 2, 2048, 200), (1000, 4, 512, 256), (777, 3, 1408, 390),
          (4000, 8, 176, 96), (2100, 1, 3328, 140), (513, 64, 320, 72)]


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_matmul(A, shape, swiglu, out):
    M, E, K, N = shape
    if swiglu and N % 2:
        N += 1
    a, b = ints(M, K, seed=M), ints(E, N, K, seed=N)
    sa = 0.5 + torch.rand(M, generator=gen(1), device="cuda")
    sb = (0.5 + torch.rand(E, N, generator=gen(2), device="cuda")) / (5000 * K ** 0.5)
    check(A, a, sa, b, sb, None if E == 1 else splits_of(E, M, M), None, swiglu, out)


@pytest.mark.parametrize("shape", [(64, 7, 8, 192, 80), (3, 24, 16, 64, 48), (700, 2000, 4, 1088, 264),
                                   (130, 130, 1, 96, 36)], ids=str)
def test_gathered_rows(A, shape):
    """rows picks (and repeats) rows of a, whose pitch is larger than K."""
    Ma, M, E, K, N = shape
    a = ints(Ma, K + 32, seed=4)[:, :K]
    rows = torch.randint(0, Ma, (M,), generator=gen(5), device="cuda").to(torch.int32)
    b = ints(E, N, K, seed=6)
    sa, sb = torch.rand(Ma, generator=gen(7), device="cuda"), torch.rand(E, N, generator=gen(8), device="cuda") / K
    sp = None if E == 1 else splits_of(E, M, 9)
    check(A, a, sa, b, sb, sp, rows, False, "bf16")
    check(A, a, sa, b, sb, sp, rows, True, "f32")


@pytest.mark.parametrize("form", ["vec", "small", "wide"])
@pytest.mark.parametrize("shape", [(1, 1, 16, 2), (33, 1, 1040, 258), (70, 3, 256, 514), (300, 5, 2048, 136),
                                   (90, 40, 4096, 64), (700, 2, 640, 1030)], ids=str)
def test_every_form(A, monkeypatch, shape, form):
    """Each form at any number of rows, plain and SwiGLU, gathered and not."""
    monkeypatch.setenv("MOE_INT8_FORM", form)
    M, E, K, N = shape
    a, b = ints(M, K, seed=M + 1), ints(E, N, K, seed=N + 1)
    sa = 0.5 + torch.rand(M, generator=gen(31), device="cuda")
    sb = (0.5 + torch.rand(E, N, generator=gen(32), device="cuda")) / (5000 * K ** 0.5)
    sp = None if E == 1 else splits_of(E, M, M + 2)
    rows = torch.randint(0, M, (M,), generator=gen(33), device="cuda").to(torch.int32)
    check(A, a, sa, b, sb, sp, None, False, "f32")
    check(A, a, sa, b, sb, sp, rows, True, "bf16")


@pytest.mark.parametrize("M", [1, 6, 200, 700])
@pytest.mark.parametrize("av,bv", [(127, 127), (-128, -128), (-128, 127), (101, 127)])
def test_extreme_sums_are_exact(A, M, av, bv):
    """Sums far beyond 2^24, and with one odd term that FP32 accumulation would lose."""
    K, N = 8192, 70
    a = torch.full((M, K), av, dtype=torch.int8, device="cuda")
    a[:, 5] = 1
    b = torch.full((1, N, K), bv, dtype=torch.int8, device="cuda")
    b[0, 1::2, 5] = 1
    one, ones = torch.ones(M, device="cuda"), torch.ones(1, N, device="cuda")
    got = A.matmul_int8(a, one, b, ones, out_dtype="f32")
    want = (a.cpu().double() @ b[0].cpu().double().T).float()  # the exact integer, rounded once
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("M", [5, 900])
def test_rows_without_an_expert_are_zero(A, M):
    a, b = ints(M, 64, seed=10), ints(3, 40, 64, seed=11)
    sp = [0, M // 5, M // 5, M // 2]
    check(A, a, torch.ones(M, device="cuda"), b, torch.ones(3, 40, device="cuda"), sp)
    check(A, a, torch.ones(M, device="cuda"), b, torch.ones(3, 40, device="cuda"), [0, 0, 0, 0])


@pytest.mark.parametrize("M", [6, 800])
def test_bad_row_index_is_reported(A, M):
    a, b = ints(10, 64, seed=12), ints(1, 24, 64, seed=13)
    rows = torch.zeros(M, dtype=torch.int32, device="cuda")
    rows[2], rows[M - 1] = 10, -1
    ws = A.alloc_int8_workspace(M, 64, 24)
    sa, sb = torch.ones(10, device="cuda"), torch.ones(1, 24, device="cuda")
    got = A.matmul_int8(a, sa, b, sb, rows=rows, out_dtype="f32", ws=ws)
    assert A.workspace_status(ws) == A.MOE_ERR_DEVICE_INDEX and A.workspace_status(ws) == A.MOE_OK
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[2] = bad[M - 1] = True
    want = (a[0].double() @ b[0].double().T).float()
    assert got[bad].isnan().all() and torch.equal(got[~bad], want.expand(M - 2, 24))
    rows[2] = rows[M - 1] = 9
    A.matmul_int8(a, sa, b, sb, rows=rows, ws=ws)
    assert A.workspace_status(ws) == A.MOE_OK


@pytest.mark.parametrize("M", [4, 600])
def test_bad_offsets_stay_in_bounds(A, M):
    """Offsets beyond the rows, descending or negative are clamped."""
    a, b = ints(M, 64, seed=14), ints(4, 32, 64, seed=15)
    sa, sb = torch.ones(M, device="cuda"), torch.ones(4, 32, device="cuda")
    for off in ([0, 2, 1, 10 * M, 99], [-5, 1, 2, 3, M + 7], [0, 2 ** 31 - 1, 0, 0, 2 ** 31 - 1]):
        out = A.matmul_int8(a, sa, b, sb, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype="f32")
        assert out.shape == (M, 32)
    torch.cuda.synchronize()


def test_nan_scales_reach_the_output(A):
    for M in (3, 600):
        a, b = ints(M, 64, seed=16), ints(1, 32, 64, seed=17)
        sa = torch.ones(M, device="cuda")
        sa[1] = math.nan
        out = A.matmul_int8(a, sa, b, torch.ones(1, 32, device="cuda"))
        assert out[1].isnan().all() and not out[[0, 2]].isnan().any()


@pytest.mark.parametrize("M", [0, 4, 700])
def test_stream_graph_and_workspace(A, M):
    K, N, E = 192, 80, 4
    a, b = ints(max(M, 1), K, seed=18)[:M], ints(E, N, K, seed=19)
    sa, sb = torch.rand(M, generator=gen(20), device="cuda"), torch.rand(E, N, generator=gen(21), device="cuda")
    off = torch.tensor([0, M // 3, M // 3, M // 2, M], dtype=torch.int32, device="cuda")
    want = A.matmul_int8(a, sa, b, sb, offsets=off, swiglu=True)
    if M == 0:
        assert want.shape == (0, 40)
        return
    ws = A.alloc_int8_workspace(M, K, N, E, swiglu=True)
    assert torch.equal(A.matmul_int8(a, sa, b, sb, offsets=off, swiglu=True, ws=ws), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = A.matmul_int8(a, sa, b, sb, offsets=off, swiglu=True, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = A.matmul_int8(a, sa, b, sb, offsets=off, swiglu=True, ws=ws)
    a.copy_(ints(M, K, seed=22))
    off.copy_(torch.tensor([0, M // 2, M // 2 + 1, M - 1, M], dtype=torch.int32))
    graph.replay()
    assert torch.equal(g, A.matmul_int8(a, sa, b, sb, offsets=off, swiglu=True))
