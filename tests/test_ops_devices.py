"""The binding of the operators around the layer refuses tensors that are not where
the call runs, before it allocates or launches. Stand-ins take the tensors' place:
the check is on the host and follows no pointer."""
import pytest
import torch

from mixture_experts_ffn_fp32_gb300 import api as A


class On:
    """What the binding asks of a CUDA tensor, on a device of the test's choice."""
    is_cuda = True

    def __init__(self, dev, dtype, *shape):
        self.dev, self.dtype, self.shape, self.of = dev, dtype, torch.Size(shape), torch.empty(shape, dtype=dtype)

    device = property(lambda self: torch.device("cuda", self.dev) if self.dev >= 0 else torch.device("cpu"))

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.of, name)


class Stream:
    cuda_stream = 0

    def __init__(self, dev):
        self.device_index = dev


F, I = torch.float32, torch.int32
CALLS = {
    "layer_norm": ([(F, 4, 8), (F, 8), (F, 8)], lambda x, w, b, **k: A.layer_norm(x, w, b, **k)),
    "layer_norm_backward": ([(F, 4, 8), (F, 4, 8), (F, 4), (F, 4), (F, 8), (torch.uint8, 999)],
                            lambda dy, x, m, r, w, ws, **k: A.layer_norm_backward(dy, x, m, r, w, ws=ws, **k)),
    "group_route": ([(F, 4, 8), (F, 8)], lambda r, b, **k: A.group_route(r, 2, bias=b, **k)),
    "group_route_backward": ([(F, 4, 2), (I, 4, 2), (F, 4, 8)], lambda d, i, r, **k: A.group_route_backward(d, i, r, **k)),
    "quantize_rows": ([(F, 4, 8)], lambda x, **k: A.quantize_rows(x, **k)),
    "matmul_int8": ([(torch.int8, 4, 16), (F, 4), (torch.int8, 2, 8, 16), (F, 2, 8), (I, 3), (I, 4), (torch.uint8, 999)],
                    lambda a, sa, b, sb, o, r, ws, **k: A.matmul_int8(a, sa, b, sb, offsets=o, rows=r, ws=ws, **k)),
}


@pytest.fixture(autouse=True)
def no_outputs(monkeypatch):
    monkeypatch.setattr(A, "_current_device", lambda: 0)

    def refuse(*a, **k):
        raise AssertionError("allocated before the check")
    monkeypatch.setattr(A, "_empty", refuse)


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_elsewhere_are_refused(name):
    specs, call = CALLS[name]
    with pytest.raises(ValueError, match="cuda:0"):  # all of them on another device than the current one
        call(*(On(1, *s) for s in specs))
    for at in range(len(specs)):  # one of them elsewhere, or on the host
        for dev in (1, -1):
            with pytest.raises(ValueError, match="cuda:0"):
                call(*(On(dev if i == at else 0, *s) for i, s in enumerate(specs)))
    with pytest.raises(ValueError, match="cuda:1"):  # a stream of another device
        call(*(On(0, *s) for s in specs), stream=Stream(1))


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_in_place_pass_the_check(name):
    specs, call = CALLS[name]
    with pytest.raises(AssertionError, match="allocated"):
        call(*(On(0, *s) for s in specs))
