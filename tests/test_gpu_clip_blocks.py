"""Clipping with factors below fp32's normal range; outputs of another shape."""
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _block
from tests._gpu import announce

def _grads(sizes, seed, scale=1.0, bf16=lambda i: i % 2 == 1):
    g = torch.Generator("cuda").manual_seed(seed)
    flat = torch.randn(sum(sizes), generator=g, device="cuda").split(sizes)
    return [(t * scale).bfloat16() if bf16(i) else t * scale for i, t in enumerate(flat)]


def _check(grads, max_norm, in_place):
    total, f, want = _block.clip(grads, max_norm)
    assert f < 1
    out = None if in_place else [torch.full_like(g, 3.0) for g in grads]
    norm, got = binding.clip_gradients(grads, max_norm, out=out)
    # fp64 sums, one rounding each of the norm, the factor and the product
    assert abs(float(norm) - total) <= 2 * _block.U32 * total
    for kind, half in ((torch.bfloat16, _block.U16), (torch.float32, _block.U32)):
        pairs = [(t.reshape(-1), w.reshape(-1)) for t, w in zip(got, want) if t.dtype == kind]
        if pairs:
            t, w = torch.cat([p[0] for p in pairs]), torch.cat([p[1] for p in pairs])
            assert _block.worst(t, w, (half + 4 * _block.U32) * w.abs() + 2.0 ** -133) <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_factors_below_the_normal_range(in_place):
    """Values far above max_norm: the factor has no fp32 value of full precision, the results have."""
    for scale, max_norm in ((1e36, 1e-3), (1e36, 1e-20), (1e30, 1e-30), (2e36, 1e-2)):
        announce(f"clip values of {scale} to {max_norm} in_place={in_place}")
        _check(_grads([5000, 70, 33], 34, scale), max_norm, in_place)
    sizes = [5000 + i if i % 97 == 0 else (37 * i) % 300 + 1 for i in range(4096)]
    _check(_grads(sizes, 35, 1e34), 1e-6, in_place)


def test_outputs_of_another_shape_are_refused():
    """The same number of elements is not enough (no GPU needed: nothing is launched)."""
    for shape, other in (((2, 3), (3, 2)), ((6,), (2, 3)), ((1, 6), (6,))):
        with pytest.raises(binding.MoELoRAError):
            binding._gradients([torch.zeros(4), torch.zeros(shape)], [torch.zeros(4), torch.zeros(other)])
    kept = binding._gradients([torch.zeros(2, 3)], [torch.zeros(2, 3)])
    assert kept[0].elements == 6


@pytest.mark.gpu
def test_outputs_of_another_shape_name_the_fault():
    g = [torch.zeros((2, 3), device="cuda"), torch.zeros(4, device="cuda")]
    with pytest.raises(binding.MoELoRAError, match="shape"):
        binding.clip_gradients(g, 1.0, out=[torch.zeros((3, 2), device="cuda"), torch.zeros(4, device="cuda")])
    with pytest.raises(binding.MoELoRAError, match="shape"):
        binding.clip_gradients(g, 1.0, out=[torch.zeros(6, device="cuda"), torch.zeros(4, device="cuda")])
