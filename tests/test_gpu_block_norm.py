"""The norms on both sides of a block, forward and backward, against float64: both
kinds, each gate, types, odd widths and pitches, rows past the registers, the calls
without a block or without a next norm."""
import itertools

import pytest
import torch

from tests import block_reference as B

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def A():
    from mixture_experts_ffn_fp32_gb300 import build
    build.build()
    from mixture_experts_ffn_fp32_gb300 import api
    return api


def rand(g, n, d, dtype=torch.float32, pad=0, scale=1.0, shift=0.0):
    return (torch.randn(n, d + pad, generator=g, device="cuda") * scale + shift).to(dtype)[:, :d]


def vector(g, d, scale=0.2, shift=0.0):
    return torch.randn(d, generator=g, device="cuda") * scale + shift


def inputs(n, d, dt, pad=0, kind="rms", gate="channel", post=True, norm=True, block=True, vectors=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer = kind == "layer"
    s = {"x": rand(g, n, d, dt, pad, 2.0, 0.5), "y": rand(g, n, d, dt, pad, 1.5, -0.3) if block else None}
    post = post and block
    s["weight"] = vector(g, d, shift=1.0) if norm and vectors else None
    s["bias"] = vector(g, d) if norm and layer and vectors else None
    s["post_weight"] = vector(g, d, shift=1.0) if post and vectors else None
    s["post_bias"] = vector(g, d) if post and layer and vectors else None
    s["gate"] = None
    if block and gate == "channel":
        s["gate"] = vector(g, d, 0.5)
    elif block and gate == "element":
        s["gate"] = rand(g, n, d, dt, pad, 0.5)
    opt = {"kind": kind, "post": post, "alpha": 1.0 if gate == "none" else 0.7}
    grads = {"dn": rand(g, n, d, dt, pad) if norm else None, "dx": rand(g, n, d, dt, pad, 0.7) if block else None}
    return s, opt, grads


def close(got, want, what):
    val, tol = want
    assert got.shape == val.shape, what
    bad = ~((got.double() - val).abs() <= tol * 1.001 + 1e-30)  # a NaN is bad
    assert not bad.any(), (what, int(bad.sum()), float(((got.double() - val).abs() - tol)[bad].max()))


def check_forward(A, s, opt, norm=True, eps=1e-5):
    got = A.block_norm(s["x"], s["y"], s["weight"], s["bias"], s["post_weight"], s["post_bias"], s["gate"],
                       norm=norm, eps=eps, **opt)
    want = B.block_norm(s["x"], s["y"], s["gate"], opt["alpha"], s["post_weight"], s["post_bias"], s["weight"],
                        s["bias"], opt["kind"] == "layer", opt["post"], norm, eps)
    assert set(got) == set(want)
    for name in want:
        close(got[name], want[name], name)
    return got


def check_backward(A, s, opt, grads, stats, x, **kw):
    got = A.block_norm_backward(x, stats, s["y"], grads["dn"], grads["dx"], s["weight"] if grads["dn"] is not None else None,
                                s["post_weight"], s["post_bias"], s["gate"], **opt, **kw)
    want = B.block_norm_backward(x, stats, s["y"], grads["dn"], grads["dx"], s["gate"], opt["alpha"], s["post_weight"],
                                 s["post_bias"], s["weight"], opt["kind"] == "layer", opt["post"])
    assert set(got) == set(want)
    for name in want:
        close(got[name], want[name], name)
    return got


def check(A, n, d, dt, pad=0, **kw):
    s, opt, grads = inputs(n, d, dt, pad, **kw)
    f = check_forward(A, s, opt, kw.get("norm", True))
    x = f["x"] if s["y"] is not None else s["x"]
    check_backward(A, s, opt, grads, f["stats"], x)


SHAPES = [(1, 1, 0), (7, 1, 3), (1, 64, 0), (33, 100, 0), (65, 256, 8), (130, 257, 0), (300, 1000, 24), (64, 1024, 0),
          (19, 1411, 5), (128, 2048, 0), (500, 2048, 1), (128, 4096, 0), (5, 8191, 0), (9, 8192, 0), (3, 12288, 0),
          (4, 16384, 0), (2, 20001, 0), (5, 16392, 0),
          # several rows a warp, the last warps part empty
          (9000, 16, 0), (5001, 33, 3), (3003, 64, 8), (4097, 128, 0), (2049, 72, 0), (700, 640, 0), (333, 5120, 0)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(A, shape, dt, kind):
    n, d, pad = shape
    check(A, n, d, DT[dt], pad, kind=kind, gate="element" if pad else "channel")


@pytest.mark.parametrize("d", [200, 1411, 4096, 20001])
@pytest.mark.parametrize("kind,gate,post,norm,vectors", list(itertools.product(
    ["rms", "layer"], ["none", "channel", "element"], [True, False], [True, False], [True, False])))
def test_forms(A, kind, gate, post, norm, vectors, d):
    check(A, 37, d, torch.bfloat16, kind=kind, gate=gate, post=post, norm=norm, vectors=vectors)


@pytest.mark.parametrize("d", [33, 768, 1411, 20001])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_without_a_block(A, kind, d):
    check(A, 41, d, torch.float16, kind=kind, block=False)
    s, opt, grads = inputs(41, d, torch.float32, kind=kind, block=False)
    f = check_forward(A, s, opt)
    grads["dx"] = torch.randn(41, d, device="cuda")  # a residual gradient joins
    check_backward(A, s, opt, grads, f["stats"], s["x"])


@pytest.mark.parametrize("d", [768, 4096])
def test_either_gradient_alone(A, d):
    s, opt, grads = inputs(60, d, torch.bfloat16, kind="layer", gate="element")
    f = check_forward(A, s, opt)
    check_backward(A, s, opt, {"dn": grads["dn"], "dx": None}, f["stats"], f["x"])
    s["weight"] = None
    check_backward(A, s, opt, {"dn": None, "dx": grads["dx"]}, f["stats"], f["x"])


def test_no_rows(A):
    s, opt, grads = inputs(0, 96, torch.float32, kind="layer")
    f = A.block_norm(s["x"], s["y"], s["weight"], s["bias"], s["post_weight"], s["post_bias"], s["gate"], **opt)
    assert f["x"].shape == f["n"].shape == (0, 96) and f["stats"].shape == (4, 0)
    got = A.block_norm_backward(f["x"], f["stats"], s["y"], grads["dn"], grads["dx"], s["weight"], s["post_weight"],
                                s["post_bias"], s["gate"], **opt)
    for name in ("dgate", "dweight", "dbias", "dpost_weight", "dpost_bias"):
        assert got[name].shape == (96,) and (got[name] == 0).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d", [96, 2048, 4096, 9000])
def test_constant_and_infinite_rows(A, d, kind):
    """Rows of zeros stay finite; a NaN or an infinity stays in its row."""
    s, opt, grads = inputs(6, d, torch.float32, kind=kind)
    s["x"], s["y"] = s["x"].contiguous(), s["y"].contiguous()
    clean = A.block_norm(**s, **opt)
    s["y"][0] = 0
    s["x"][0] = 0
    s["y"][2, 3] = float("nan")
    s["x"][4, d - 1] = float("inf")
    got = A.block_norm(**s, **opt)
    assert got["x"][0].isfinite().all() and got["n"][0].isfinite().all()
    assert got["n"][2].isnan().all() and got["n"][4].isnan().any()
    for name in ("x", "n"):
        assert torch.equal(got[name][[1, 3, 5]], clean[name][[1, 3, 5]])


def test_large_mean(A):
    s, opt, grads = inputs(16, 2048, torch.float32, kind="layer")
    s["y"] = (s["y"] + 4096.0).contiguous()
    check_forward(A, s, opt)


def test_against_differences(A):
    """Every gradient against central differences of the float64 forward."""
    n, d, eps, h = 3, 40, 1e-3, 1e-6
    for kind, gate in itertools.product(["rms", "layer"], ["channel", "element"]):
        s, opt, grads = inputs(n, d, torch.float32, kind=kind, gate=gate)
        f = A.block_norm(**s, **opt, eps=eps)
        got = A.block_norm_backward(f["x"], f["stats"], s["y"], grads["dn"], grads["dx"], s["weight"],
                                    s["post_weight"], s["post_bias"], s["gate"], **opt)
        v = {k: t.double() for k, t in s.items() if t is not None}

        def loss(v):
            r = B.block_norm(v["x"], v["y"], v["gate"], opt["alpha"], v["post_weight"], v.get("post_bias"), v["weight"],
                             v.get("bias"), kind == "layer", True, True, eps)
            return float((r["n"][0] * grads["dn"].double()).sum() + (r["x"][0] * grads["dx"].double()).sum())
        B.HALF[torch.float64], B.TINY[torch.float64] = 0.0, 0.0
        names = {"x": "dx", "y": "dy", "gate": "dgate", "weight": "dweight", "bias": "dbias",
                 "post_weight": "dpost_weight", "post_bias": "dpost_bias"}
        for name, t in v.items():
            for at in (0, t.numel() // 2, t.numel() - 1):
                up, dn = dict(v), dict(v)
                up[name], dn[name] = t.clone(), t.clone()
                up[name].view(-1)[at] += h
                dn[name].view(-1)[at] -= h
                diff = (loss(up) - loss(dn)) / (2 * h)
                # the difference itself is good to about 1e-9 / h
                assert abs(float(got[names[name]].reshape(-1)[at]) - diff) <= 2e-4 * max(1.0, abs(diff)), (kind, gate, name)


def test_strides_streams_and_graphs(A):
    """A captured forward and backward replay on new inputs; a side stream gives the same bits."""
    s, opt, grads = inputs(200, 1024, torch.bfloat16, 8, gate="element")
    eager = A.block_norm(**s, **opt)
    back = A.block_norm_backward(eager["x"], eager["stats"], s["y"], **grads, weight=s["weight"],
                                 post_weight=s["post_weight"], gate=s["gate"], **opt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = A.block_norm(**s, **opt, stream=side)
    back2 = A.block_norm_backward(there["x"], there["stats"], s["y"], **grads, weight=s["weight"],
                                  post_weight=s["post_weight"], gate=s["gate"], **opt, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for k in eager:
        assert torch.equal(eager[k], there[k])
    for k in back:
        assert torch.equal(back[k], back2[k])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = A.block_norm(**s, **opt)
        b = A.block_norm_backward(f["x"], f["stats"], s["y"], **grads, weight=s["weight"],
                                  post_weight=s["post_weight"], gate=s["gate"], **opt)
    s["x"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    again = A.block_norm(**s, **opt)
    want = A.block_norm_backward(again["x"], again["stats"], s["y"], **grads, weight=s["weight"],
                                 post_weight=s["post_weight"], gate=s["gate"], **opt)
    for k in again:
        assert torch.equal(f[k], again[k])
    for k in want:
        assert torch.equal(b[k], want[k])


def test_bits_repeat(A):
    s, opt, grads = inputs(3001, 768, torch.float16, kind="layer")
    f = A.block_norm(**s, **opt)
    runs = [A.block_norm_backward(f["x"], f["stats"], s["y"], **grads, weight=s["weight"], post_weight=s["post_weight"],
                                  post_bias=s["post_bias"], gate=s["gate"], **opt) for _ in range(2)]
    for k in runs[0]:
        assert torch.equal(runs[0][k], runs[1][k])


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("kind,gate,post", [("rms", "element", True), ("layer", "element", True), ("layer", "channel", False),
                                            ("rms", "element", False)])
def test_part_empty_warps_after_nans(A, kind, gate, post, dt):
    """Rows that a warp's part has no row for add nothing, whatever an earlier kernel left in shared memory."""
    nan = float("nan")
    for n, d in ((1, 16), (5, 16), (66, 16), (850, 16), (3, 33), (66, 32), (13, 64), (47, 6), (2, 100), (9, 128), (335, 128)):
        s, opt, grads = inputs(n, d, DT[dt], kind=kind, gate=gate, post=post)
        f = A.block_norm(s["x"], s["y"], s["weight"], s["bias"], s["post_weight"], s["post_bias"], s["gate"], **opt)
        left, _, lgrads = inputs(16384, d, DT[dt], kind=kind, gate="element", post=post, vectors=False)
        left = {k: None if v is None else torch.full_like(v, nan) for k, v in {**left, **lgrads}.items()}
        stats = torch.full((4 if kind == "layer" else 2, 16384), nan, device="cuda")
        # without the vectors' gradients the last kernel is the one that keeps rows in shared memory
        A.block_norm_backward(left["x"], stats, left["y"], left["dn"], left["dx"], gate=left["gate"], weight_grads=False, **opt)
        torch.cuda.synchronize()
        check_backward(A, s, opt, grads, f["stats"], f["x"])


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("n,d,pad", [(3, 6, 2), (33, 100, 4), (40, 96, 8), (9, 1003, 5), (70, 2040, 8), (3, 8190, 2), (2, 16392, 8)])
def test_nans_between_rows(A, n, d, pad, kind, dt):
    """What lies between a row's end and its pitch reaches no result."""
    s, opt, grads = inputs(n, d, DT[dt], kind=kind, gate="element")
    for group in (s, grads):
        for k, v in group.items():
            if v is not None and v.dim() == 2:
                whole = torch.full((n, d + pad), float("nan"), device="cuda", dtype=v.dtype)
                whole[:, :d] = v
                group[k] = whole[:, :d]
    f = check_forward(A, s, opt)
    check_backward(A, s, opt, grads, f["stats"], f["x"])
