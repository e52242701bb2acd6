"""The forms of the 8-bit expert products against each other: the sums are exact
in all of them, and the scales and SiLU are the same operations in the same order,
so outputs are equal bit for bit, whichever form a call's sizes take."""
import pytest
import torch

from tests.test_gpu_int8 import A, DT, gen, ints, splits_of  # noqa: F401

pytestmark = pytest.mark.gpu
FORMS = ["vec", "small", "wide"]


def forms(A, monkeypatch, *args, **kw):  # noqa: F811
    got = {}
    for form in FORMS:
        monkeypatch.setenv("MOE_INT8_FORM", form)
        got[form] = A.matmul_int8(*args, **kw)
    return got


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 16, 2), (37, 1, 1040, 258), (90, 5, 256, 512), (300, 4, 2048, 136), (600, 2, 640, 1030)],
                         ids=str)
def test_forms_agree_bit_for_bit(A, monkeypatch, shape, swiglu, out):  # noqa: F811
    """Scales that are no powers of two; gates from far below zero to far above."""
    M, E, K, N = shape
    a, b = ints(M, K, seed=M), ints(E, N, K, seed=N)
    sa = (0.1 + torch.rand(M, generator=gen(1), device="cuda")) * 20 ** torch.rand(M, generator=gen(2), device="cuda")
    sb = (0.5 + torch.rand(E, N, generator=gen(3), device="cuda")) / (2000 * K ** 0.5)
    sp = splits_of(E, M, M)
    off = None if E == 1 else torch.tensor(sp, dtype=torch.int32, device="cuda")
    rows = torch.randint(0, M, (M,), generator=gen(4), device="cuda").to(torch.int32)
    got = forms(A, monkeypatch, a, sa, b, sb, offsets=off, rows=rows, swiglu=swiglu, out_dtype=out)
    bits = torch.int32 if out == "f32" else torch.int16
    assert (got["vec"] != 0).any()
    for form in FORMS[1:]:
        assert torch.equal((got[form] + 0.0).view(bits), (got["vec"] + 0.0).view(bits)), form


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gates_far_below_zero(A, monkeypatch, form, out):  # noqa: F811
    """Gates from -95 to 0 with ups of 1e30: SiLU(gate) below FP32's normal range still counts."""
    monkeypatch.setenv("MOE_INT8_FORM", form)
    K, F, M = 64, 96, 40
    a = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    a[:, 0] = 1
    b = torch.zeros(1, 2 * F, K, dtype=torch.int8, device="cuda")
    b[0, :F, 0] = -torch.arange(F, device="cuda").to(torch.int8)
    b[0, F:, 0] = 1
    sb = torch.ones(1, 2 * F, device="cuda")
    sb[0, F:] = 1e30
    sa = torch.linspace(0.9, 1.0, M, device="cuda")
    got = A.matmul_int8(a, sa, b, sb, swiglu=True, out_dtype=out)
    g = -(sa.double()[:, None] * torch.arange(F, device="cuda").double())
    want = g * torch.sigmoid(g) * (sa.double() * sb[0, F].double())[:, None]
    # five roundings of the scales and products, the sigmoid's 8 half steps and its argument's g; below
    # exp(-87.3) the exponential is a multiple of 2^-149, half of which it may be off by
    rel = 2.0 ** -24 * (16 + 4 * g.abs()) + 2.0 ** -150 / torch.sigmoid(g) * 2
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[out]
    assert ((got.double() - want).abs() <= (rel + half * 1.001) * want.abs()).all()
