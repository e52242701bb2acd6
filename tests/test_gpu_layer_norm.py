"""Layer norm forward and backward against float64, over types, odd widths,
strided rows, single rows and columns, and large means."""
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


def rand(shape, seed, scale=1.0, dtype=torch.float32, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(shape[0], shape[1] + pad, generator=g, device="cuda") * scale
    return t.to(dtype)[:, :shape[1]]


# rows, width, pad of the pitch: one element, one column, warp rows, each CTA
# width, odd widths, unaligned pitches, rows past the register forms
SHAPES = [(1, 1, 0), (7, 1, 3), (1, 64, 0), (33, 100, 0), (65, 256, 8), (130, 257, 0), (300, 1000, 24), (64, 1024, 0),
          (19, 1411, 5), (128, 2048, 0), (1000, 2048, 1), (128, 4096, 0), (5, 8191, 0), (9, 8192, 0), (3, 12288, 0),
          (4, 16384, 0), (2, 20001, 0), (5, 16392, 0),
          # several rows a warp, the last warps part empty
          (9000, 16, 0), (5001, 33, 3), (3003, 64, 8), (4097, 128, 0), (2049, 72, 0)]


def check_forward(x, w, b, eps, got):
    y, mu, rstd, xh = R.layer_norm(x, w, b, eps)
    d = x.shape[1]
    xd = x.double()
    # sums of d terms in chains of at most 16 (long rows: d / 1024) and a tree of 10
    n = 26 + d / 1024
    mag = xd.abs().mean(1)
    gam = 1.0 if w is None else w.double().abs()
    bet = 0.0 if b is None else b.double().abs()
    var = rstd ** -2
    # the mean: first estimate off by n U mag, corrected by the residual's mean, rounded
    assert ((got["mean"].double() - mu).abs() <= R.U * (2 * mu.abs() + n * var.sqrt()) + n * n * R.U ** 2 * mag).all()
    assert ((got["rstd"].double() - rstd).abs() <= R.U * (n + 8) * rstd + 1e-3 * R.U * rstd).all()
    core = R.U * ((n + 12) * xh.abs() + n) + 2 * R.U * (n * n * R.U * mag * rstd)[:, None]
    # x less the first mean rounds once, by what it is
    tol = R.HALF[x.dtype] * y.abs() + gam * (core + 2 * R.U * xh.abs()) + R.U * bet
    assert ((got["y"].double() - y).abs() <= tol * 1.001 + 1e-30 + (6e-8 if x.dtype == torch.float16 else 0)).all()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(A, shape, dt):
    n, d, pad = shape
    x = rand((n, d), 1, 2.0, DT[dt], pad) + 0.5
    x = x if pad == 0 else rand((n, d), 1, 2.0, DT[dt], pad)
    w, b = rand((1, d), 2)[0].contiguous(), rand((1, d), 3)[0].contiguous()
    check_forward(x, w, b, 1e-5, A.layer_norm(x, w, b, 1e-5))


@pytest.mark.parametrize("w,b", [(True, False), (False, True), (False, False)])
def test_without_weight_or_bias(A, w, b):
    x = rand((40, 384), 4)
    w = rand((1, 384), 5)[0].contiguous() if w else None
    b = rand((1, 384), 6)[0].contiguous() if b else None
    check_forward(x, w, b, 1e-3, A.layer_norm(x, w, b, 1e-3))


@pytest.mark.parametrize("d", [96, 1024, 2048, 5000])
def test_mean_large_against_deviation(A, d):
    x = rand((16, d), 7) + 4096.0
    check_forward(x, None, None, 1e-5, A.layer_norm(x, None, None, 1e-5))


def test_constant_rows_and_nan(A):
    x = torch.full((4, 640), 3.25, device="cuda")
    got = A.layer_norm(x, None, None, 1e-5)
    assert (got["y"] == 0).all() and (got["mean"] == 3.25).all()
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    got = A.layer_norm(x)
    assert got["y"][1].isnan().all() and got["rstd"][1].isnan() and got["y"][2].isnan().any()
    assert (got["y"][[0, 3]] == 0).all()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(A, shape, dt):
    n, d, pad = shape
    x, dy = rand((n, d), 8, 1.5, DT[dt], pad), rand((n, d), 9, 1.0, DT[dt], pad)
    w = 1 + 0.2 * rand((1, d), 10)[0].contiguous()
    _, mu, rstd, _ = R.layer_norm(x, w, None, 1e-2)
    mu, rstd = mu.float(), rstd.float()
    got = A.layer_norm_backward(dy, x, mu, rstd, w)
    dx, dw, db, xh, g = R.layer_norm_backward(dy, x, mu, rstd, w)
    k = 26 + d / 1024
    rs = rstd.double()[:, None]
    parts = g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)
    tol = R.HALF[x.dtype] * dx.abs() + R.U * (k + 12) * rs * parts
    assert ((got["dx"].double() - dx).abs() <= tol + (6e-8 if dt == "f16" else 0)).all()
    # a column's sum: n terms, each off by 4 U, in chains that no order makes longer than n
    chain = min(n, n / 100 + 60) + 5
    assert ((got["dbias"].double() - db).abs() <= R.U * chain * dy.double().abs().sum(0)).all()
    assert ((got["dweight"].double() - dw).abs() <= R.U * (chain + 4) * (dy.double() * xh).abs().sum(0)).all()


def test_backward_against_differences(A):
    """dx, dweight and dbias against central differences of the float64 forward."""
    n, d = 3, 40
    x, dy = rand((n, d), 11), rand((n, d), 12)
    w, b = rand((1, d), 13)[0].contiguous(), rand((1, d), 14)[0].contiguous()
    f = A.layer_norm(x, w, b, 1e-5)
    got = A.layer_norm_backward(dy, x, f["mean"], f["rstd"], w)
    h = 1e-6

    def loss(x, w, b):
        return float((R.layer_norm(x, w, b, 1e-5)[0] * dy.double()).sum())

    for name, base, grad in (("x", x.double(), got["dx"]), ("w", w.double(), got["dweight"]),
                             ("b", b.double(), got["dbias"])):
        flat = base.reshape(-1)
        for i in range(0, flat.numel(), 7):
            up, dn = flat.clone(), flat.clone()
            up[i] += h
            dn[i] -= h
            args = {"x": x.double(), "w": w.double(), "b": b.double()}
            hi = loss(**{**args, name: up.view_as(base)})
            lo = loss(**{**args, name: dn.view_as(base)})
            # differences: 1e-9 from h^2, 1e-9 from cancellation; gradients: FP32
            assert abs((hi - lo) / (2 * h) - float(grad.reshape(-1)[i])) < 2e-5


def test_backward_parts(A):
    x, dy = rand((50, 512), 15), rand((50, 512), 16)
    f = A.layer_norm(x)
    full = A.layer_norm_backward(dy, x, f["mean"], f["rstd"])
    only = A.layer_norm_backward(dy, x, f["mean"], f["rstd"], weight_grads=False)
    assert set(only) == {"dx"} and torch.equal(only["dx"], full["dx"])
    again = A.layer_norm_backward(dy, x, f["mean"], f["rstd"])
    assert all(torch.equal(full[k], again[k]) for k in full)


def test_no_rows(A):
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    n0 = A.launch_count()
    f = A.layer_norm(x)
    assert f["y"].shape == (0, 64) and A.launch_count() == n0
    g = A.layer_norm_backward(x, x, f["mean"], f["rstd"])
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_stream_and_graph(A):
    x, dy = rand((256, 1024), 17, dtype=torch.bfloat16), rand((256, 1024), 18, dtype=torch.bfloat16)
    want = A.layer_norm(x)
    wb = A.layer_norm_backward(dy, x, want["mean"], want["rstd"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = A.layer_norm(x, stream=s)
    gb = A.layer_norm_backward(dy, x, got["mean"], got["rstd"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got["y"], want["y"]) and all(torch.equal(gb[k], wb[k]) for k in wb)
    graph = torch.cuda.CUDAGraph()
    x2, dy2 = x.clone(), dy.clone()
    with torch.cuda.graph(graph):
        f = A.layer_norm(x2)
        b = A.layer_norm_backward(dy2, x2, f["mean"], f["rstd"])
    x2.copy_(dy)
    dy2.copy_(x)
    graph.replay()
    want = A.layer_norm(dy)
    wb = A.layer_norm_backward(x, dy, want["mean"], want["rstd"])
    assert torch.equal(f["y"], want["y"]) and all(torch.equal(b[k], wb[k]) for k in wb)


# CTAs of three quarters of a power of two, whole and part full, several rows each
THREE_QUARTERS = [(40, 1280, 0), (1301, 1536, 8), (1001, 2560, 0), (700, 2561, 1), (505, 5120, 8), (161, 5121, 0),
                  (320, 6144, 0)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", THREE_QUARTERS, ids=str)
def test_three_quarter_widths(A, shape, dt):
    test_forward(A, shape, dt)
    test_backward(A, shape, dt)


# 4 to 16 columns a thread, 8 to 128 threads a row; rows that end inside a warp's
SHORT_ROWS = [(5003, 1411, 5), (3000, 1100, 3), (2900, 257, 0), (777, 384, 3),
              (9001, 26, 0), (4100, 17, 3), (1, 2, 0), (6007, 47, 0), (3003, 114, 8), (2050, 99, 1), (5146, 163, 0),
              (2500, 160, 0), (3460, 320, 0), (1501, 333, 0), (900, 576, 3), (1001, 777, 0)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHORT_ROWS, ids=str)
def test_short_rows(A, shape, dt):
    test_forward(A, shape, dt)
    test_backward(A, shape, dt)
