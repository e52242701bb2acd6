"""Low-rank adapters of small whole numbers over wide inputs: every product and sum, in any order and in
pieces, is a whole number that FP32 has, so results are equal to the last bit; an element of d, a rank or a
slice that a kernel left out or took twice shows."""
import pytest
import torch

from tests.test_gpu_adapter import A, DT, form, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("T,d,N,r,E", [(1, 4096, 2048, 16, 8), (33, 8192, 64, 48, 4), (5, 8200, 72, 16, 2), (40, 8191, 61, 12, 3),
                                       (300, 5000, 200, 40, 3), (600, 8192, 520, 24, 2), (900, 8192, 128, 128, 2), (2100, 4104, 136, 64, 3),
                                       (64, 2056, 1100, 256, 2)])
def test_whole_numbers(A, form, T, d, N, r, E, dt, out):  # noqa: F811
    s = make(T, d, N, r, E, DT[dt], DT[out])
    g = torch.Generator(device="cuda").manual_seed(1)

    def whole(top, *shape):
        return torch.randint(-top, top + 1, shape, generator=g, device="cuda")
    x, a, b, base = whole(1, T, d), whole(1, E, r, d), whole(1, E, N, r), whole(100, T, N)
    # v is at most 8200, or 2^14 twice, and its sums at most 256 times that: below 2^24 (BF16's pieces have 16 bits)
    s.update(x=x.to(DT[dt]), a=a.to(DT[dt]), b=b.to(DT[dt]), base=base.to(DT[out]), scale=torch.full((E,), 2.0, device="cuda"))
    want = base.double()
    off = s["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        at = s["rows"][lo:hi].long()
        want[at] += 2 * (x[at].double() @ a[e].double().T) @ b[e].double().T
    assert want.abs().max() < 1 << 24
    want = want.float().to(DT[out]) if DT[out] != torch.float16 else want.clamp(-65504, 65504).float().half()
    got = A.adapter_add(**s)
    assert torch.equal(got, want)
