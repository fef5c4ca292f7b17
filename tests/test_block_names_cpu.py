"""Names that block_norm_backward does not know are refused, not passed over (no GPU
needed: nothing is launched)."""
import pytest
import torch

from mixture_experts_layer_up_amd import binding


@pytest.mark.parametrize("kw", [dict(wanted=("residual", "pre")), dict(wanted=["d_branch"]),
                                dict(out={"d_residual": torch.zeros(4, 64)}), dict(wanted="residual"),
                                dict(out={"residual": torch.zeros(4, 64), "normed": torch.zeros(4, 64)})])
def test_unknown_gradients(kw):
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    shape = binding.NormShape(4, 64, 1e-6, 1.0, 0.0, 0)
    with pytest.raises(binding.MoELoRAError, match="gradients are named"):
        binding.block_norm_backward(shape, x, x, pre_weight=w, d_residual=x, d_normed=x, **kw)
