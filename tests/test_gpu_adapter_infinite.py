"""Infinities in low-rank adapters' B (and in x beside them) against the formula in 64
bits: an infinite product is an infinity, of the right sign, and NaN only where the formula
has one (infinities of both signs, zero times infinity)."""
import pytest
import torch

from tests import block_reference as B
from tests.test_gpu_adapter import A, DT, form, make  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")


def check(got, s):
    T, d = s["x"].shape
    clean = {**s, "x": s["x"].nan_to_num(0, 0, 0), "b": s["b"].nan_to_num(0, 0, 0)}
    val, tol = B.adapter_add(clean["base"], clean["x"], clean["a"], clean["b"], s["offsets"], s["rows"], s["scale"], got.dtype,
                             2 if got.dtype != torch.float32 else 3)
    want = s["base"].double().clone()
    finite = torch.ones_like(want, dtype=torch.bool)
    off = s["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        at = s["rows"][lo:hi].long()
        v = float(s["scale"][e]) * (s["x"][at].double()[:, None, :] * s["a"][e].double()).sum(2)
        p = v[:, None, :] * s["b"][e].double()
        want[at] += p.sum(2)
        finite[at] = p.isfinite().all(2)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.double()[~finite & ~want.isnan()], want[~finite & ~want.isnan()])
    assert ((got.double() - val).abs() <= tol * 1.001 + 1e-30)[finite].all()
    return want


@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("T,d,N,r", [(1, 64, 72, 16), (50, 264, 136, 16), (50, 264, 136, 64), (70, 100, 61, 12), (40, 72, 104, 96),
                                     (300, 128, 200, 40), (900, 96, 328, 128)])
def test_infinite_b(A, form, T, d, N, r, dt, out):  # noqa: F811
    s = make(T, d, N, r, 3, DT[dt], DT[out], ids=torch.arange(T) % 4)
    b = s["b"]
    b[0, 3, 1], b[0, N - 1, r - 1] = INF, -INF          # alone in their columns
    b[0, 9, 2] = b[0, 9, r - 2] = INF                    # two in one: an infinity or NaN by the signs of v
    b[1, :, 0] = INF                                     # every column
    b[2, 5] = -INF                                       # every rank
    b[2, 7, 0] = float("nan")
    want = check(A.adapter_add(**s), s)
    assert want.isinf().any() and (T == 1 or want.isnan().any())
    got = A.adapter_add(**s, out=s["base"].clone())
    assert torch.equal(got.isnan(), want.isnan())
    inplace = A.adapter_add(**{**s, "base": (own := s["base"].clone())}, out=own)
    assert torch.equal(inplace.nan_to_num(7.0), got.nan_to_num(7.0))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,d,N,r", [(50, 264, 136, 16), (70, 100, 61, 12), (900, 96, 328, 64)])
def test_infinite_x_and_b(A, form, T, d, N, r, dt):  # noqa: F811
    """Rows of zeros, with an infinity and with a NaN against infinite and zero elements of B."""
    s = make(T, d, N, r, 2, DT[dt], torch.float32, ids=torch.arange(T) % 3)
    s["b"][0, 4, 1], s["b"][1, :, r - 1] = INF, -INF
    s["b"][0, 6, 0] = 0
    for i, v in ((0, 0.0), (4, 0.0)):
        s["x"][i] = v
    s["x"][3, 5], s["x"][6, d - 1], s["x"][9, 0] = INF, -INF, float("nan")
    s["a"].abs_()
    check(A.adapter_add(**s), s)
