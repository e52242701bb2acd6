"""The configs that the operators' binding keeps are keyed by values."""
import torch

from mixture_experts_ffn_fp32_gb300 import api as A


def test_scale_is_taken_by_value():
    """A scale held in a tensor that changes between two calls."""
    logits, scale = torch.zeros(2, 8), torch.tensor(1.5)

    def config():
        return A._group_config(logits, 2, 1, 1, 2, "sigmoid", True, scale)._obj
    assert config().scale == 1.5
    scale.fill_(2.5)
    assert config().scale == 2.5
    assert A._group_config(logits, 2, 1, 1, 2, "sigmoid", True, 2)._obj.scale == 2.0
