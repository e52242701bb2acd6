"""FP32 outputs of 16-bit adapters: the low bits of the inner values count where they add up
behind a large sum."""
import pytest
import torch

from tests.test_gpu_adapter import A, DT, form, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("r", [48, 96, 128, 256])
@pytest.mark.parametrize("T,N", [(1, 64), (40, 136), (40, 61), (300, 264), (300, 61)])
def test_low_bits_of_later_ranks(A, form, T, N, r, dt):  # noqa: F811
    """v is 1/2 in the first 16 ranks (b 1: together 8), then 2^-10 + b 2^-24 with b 1 and -1 in turn: the large
    parts cancel exactly, the small ones add up to (r - 16) 2^-24, a whole number of units of 8 (2^-20) that
    FP32 has. Every partial sum of either part by itself is exact, so the sum of both is. (FP32 operands have no
    parts: each 2^-24 is lost by itself, at most half a unit each.)"""
    s = make(T, 64, N, r, 2, DT[dt], torch.float32, ids=torch.arange(T) % 2)
    k = torch.arange(r, device="cuda")
    sign = torch.where(k < 16, 1.0, torch.where(k % 2 == 0, 1.0, -1.0))
    s["x"].zero_()
    s["x"][:, :2] = 1
    s["a"].zero_()
    s["a"][:, :, 0] = torch.where(k < 16, 0.5, 2.0 ** -10)
    s["a"][:, :, 1] = torch.where(k < 16, 0.0, sign * 2.0 ** -24)
    s["b"].copy_(sign.expand(2, N, r))
    s["scale"] = s["base"] = None
    s["x"][::3] *= -1
    got = A.adapter_add(**s, out=torch.empty(T, N, device="cuda"))
    want = 8 + (r - 16) * 2.0 ** -24
    want = torch.where(torch.arange(T, device="cuda") % 3 == 0, -want, want)[:, None].expand(T, N)
    if dt == "f32":
        assert ((got - want).abs() <= (r - 16) * 2.0 ** -21).all()
    else:
        assert torch.equal(got, want)
