"""The binding refuses a workspace whose number of elements is not what lies in memory:
one of strided or of repeated bytes."""
import pytest
import torch

from mixture_experts_ffn_fp32_gb300 import api as A
from tests.test_ops_devices import CALLS, On, no_outputs  # noqa: F401

F, H, I, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
WITH = {n: CALLS[n] for n in ("layer_norm_backward", "matmul_int8")}
WITH["block_norm_backward"] = ([(H, 4, 8), (F, 2, 4), (H, 4, 8), (H, 4, 8), (U8, 9999)],
                               lambda x, st, y, dn, ws: A.block_norm_backward(x, st, y, dn, ws=ws))
WITH["adapter_add"] = ([(H, 4, 8), (H, 3, 2, 8), (H, 3, 6, 2), (I, 4), (U8, 9999)],
                       lambda x, a, b, o, ws: A.adapter_add(None, x, a, b, o, ws=ws))


@pytest.mark.parametrize("name", list(WITH))
@pytest.mark.parametrize("odd", [lambda t: t[::2], lambda t: t[:1].expand(1 << 20), lambda t: t.view(-1, 9)[:, :8]])
def test_strided_workspaces_are_refused(name, odd):
    specs, call = WITH[name]
    args = [On(0, *s) for s in specs]
    args[-1].of = odd(torch.empty(9999, dtype=U8))
    with pytest.raises(ValueError, match="contiguous"):
        call(*args)
