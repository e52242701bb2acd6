"""Adapters of ranks at which a kernel's shared memory leaves one CTA an SM, from one row to many,
narrow and wide inputs: CTAs of a tile with and without a part of d."""
import pytest

from tests.test_gpu_adapter import A, DT, check, form, make  # noqa: F401

import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("T,d,N,r,E", [(1, 2048, 2048, 256, 4), (64, 2048, 2056, 128, 16), (300, 1024, 520, 256, 128), (1000, 512, 264, 256, 32),
                                       (129, 8, 64, 128, 1), (400, 64, 136, 112, 3), (2000, 72, 256, 104, 2), (9000, 1100, 128, 128, 70),
                                       (45000, 128, 64, 112, 2)])
def test_large_ranks(A, form, T, d, N, r, E, dt, out):  # noqa: F811
    s = make(T, d, N, r, E, DT[dt], DT[out])
    got = A.adapter_add(**s)
    check(got, s)
    assert torch.equal(got, A.adapter_add(**s))
