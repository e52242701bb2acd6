"""Row indices of low-rank adapters that name no row, in every form and type: skipped,
reported, and no other row touched, with an adapter or without one."""
import pytest
import torch

from tests.test_gpu_adapter import A, DT, form, make  # noqa: F401

pytestmark = pytest.mark.gpu


def case(dt, T, behind):
    """A third of the rows without an adapter; one bad index among those (behind), or before them."""
    s = make(T, 128, 192, 16, 3, DT[dt], ids=torch.arange(T) % 4)
    first = int(s["offsets"][3])
    at = [first, T - 1, (first + T) // 2] if behind else [0, first - 1]
    lost = s["rows"][at].long()
    return s, at, lost


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T", [5, 60, 3000])
@pytest.mark.parametrize("behind", [True, False])
@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_bad_rows_are_reported(A, form, dt, T, behind, bad):  # noqa: F811
    s, at, lost = case(dt, T, behind)
    ws = A.alloc_adapter_workspace(T, 128, 192, 16, 3, DT[dt])
    want = A.adapter_add(**s, ws=ws)
    assert A.workspace_status(ws) == A.MOE_OK
    for i in at:  # one at a time: each by itself is reported
        out = torch.full_like(want, 7.0)
        rows = s["rows"].clone()
        rows[i] = bad
        A.adapter_add(**{**s, "rows": rows}, out=out, ws=ws)
        assert A.workspace_status(ws) == A.MOE_ERR_DEVICE_INDEX and A.workspace_status(ws) == A.MOE_OK
        row = int(s["rows"][i])
        assert (out[row] == 7).all()
        keep = torch.arange(T, device="cuda") != row
        assert torch.equal(out[keep], want[keep])


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T", [5, 60, 3000])
def test_in_place(A, form, dt, T):  # noqa: F811
    """Rows without an adapter stay as they are, and their positions are not looked at; the others' are."""
    s, at, lost = case(dt, T, True)
    ws = A.alloc_adapter_workspace(T, 128, 192, 16, 3, DT[dt])
    want, base = A.adapter_add(**s), s["base"].clone()
    s["rows"][at] = -5
    got = A.adapter_add(**s, out=s["base"], ws=ws)
    assert A.workspace_status(ws) == A.MOE_OK and torch.equal(got, want)
    s["base"].copy_(base)
    first = int(s["rows"][0])
    s["rows"][0] = T
    got = A.adapter_add(**s, out=s["base"], ws=ws)
    assert A.workspace_status(ws) == A.MOE_ERR_DEVICE_INDEX
    assert torch.equal(got[first], base[first])
    keep = torch.arange(T, device="cuda") != first
    assert torch.equal(got[keep], want[keep])
