"""moe_lora_clip_gradients on the GPU against float64."""
import math

import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _block
from tests._gpu import announce

pytestmark = pytest.mark.gpu


def _grads(sizes, seed=1, scale=1.0, kinds=("f", "b")):
    g = torch.Generator("cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n, generator=g, device="cuda") * scale
        out.append(t.bfloat16() if kinds[i % len(kinds)] == "b" else t)
    return out


def _check(grads, max_norm, in_place=False, out=None):
    total, f, want = _block.clip(grads, max_norm)
    kept = [g.clone() for g in grads]
    if not in_place and out is None:
        out = [torch.full_like(g, 3.0) for g in grads]
    norm, got = binding.clip_gradients(grads, max_norm, out=out)
    # fp64 sums, one rounding each of the norm, the factor and the product
    assert abs(float(norm) - total) <= 2 * _block.U32 * total
    for g, k, t, w in zip(grads, kept, got, want):
        half = _block.U16 if t.dtype == torch.bfloat16 else _block.U32
        bound = (half + 4 * _block.U32) * w.abs() + 2.0 ** -133     # or half a step below the normal range
        assert _block.worst(t, w, bound) <= 1
        assert in_place or torch.equal(g, k)
    return float(norm), f


SIZES = [1, 2, 7, 8, 9, 63, 1000, 32767, 32768, 32769, 100003]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kinds", ["f", "b", "fb"])
def test_sizes(kinds, in_place):
    announce(f"clip sizes {kinds} in_place={in_place}")
    _check(_grads(SIZES, kinds=kinds), 1.5, in_place)
    _check(_grads(SIZES, kinds=kinds), 1e6, in_place)


@pytest.mark.parametrize("count", [1, 111, 112, 113, 225, 1000])
def test_counts(count):
    """Tables of up to 112 tensors a launch; empty tensors among them."""
    announce(f"clip {count} tensors")
    g = _grads([(37 * i) % 500 for i in range(1, count + 1)], seed=2)
    if count > 1:
        assert any(t.numel() == 0 for t in g) or count < 500
    _check(g, 0.25)
    _check(g, 0.25, in_place=True)


def test_views_at_every_offset():
    """Tensors that begin at any element, outputs at other offsets than inputs."""
    announce("clip offsets")
    for kind in (torch.float32, torch.bfloat16):
        buf = torch.randn(40000, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(kind)
        res = torch.zeros(40000, dtype=kind, device="cuda")
        cuts = [0] + [i * 4000 + i for i in range(1, 10)]
        grads = [buf[a:b] for a, b in zip(cuts, cuts[1:])]
        _check(grads, 2.0, out=[res[a:b] for a, b in zip(cuts, cuts[1:])])
        _check(grads, 2.0, out=[res[a + 5:b + 5] for a, b in zip(cuts, cuts[1:])])
        assert not res[cuts[-1] + 5:].any()
        tail = buf[cuts[-1]:].clone()
        _check(grads, 2.0, in_place=True)
        assert torch.equal(buf[cuts[-1]:], tail)


def test_shapes_and_zeros():
    announce("clip zeros")
    g = [torch.zeros((3, 5), device="cuda"), torch.zeros((), device="cuda"), torch.zeros((2, 0), device="cuda")]
    norm, out = binding.clip_gradients(g, 1.0)
    assert float(norm) == 0 and all(o is t for o, t in zip(out, g)) and not any(o.any() for o in out)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_norms_that_are_not_finite(bad):
    """The values stay as they are, in place and into another tensor."""
    announce(f"clip {bad}")
    g = _grads([1000, 40000, 33], seed=4)
    g[1][777] = bad
    kept = [t.clone() for t in g]
    out = [torch.zeros_like(t) for t in g]
    norm, _ = binding.clip_gradients(g, 0.5, out=out)
    assert not math.isfinite(float(norm))
    for t, k, o in zip(g, kept, out):
        assert torch.equal(t.nan_to_num(1, 2, 3), k.nan_to_num(1, 2, 3))
        assert torch.equal(o.nan_to_num(1, 2, 3), k.nan_to_num(1, 2, 3))
    binding.clip_gradients(g, 0.5)
    assert all(torch.equal(t.nan_to_num(1, 2, 3), k.nan_to_num(1, 2, 3)) for t, k in zip(g, kept))


def test_values_whose_squares_leave_fp32():
    """1e30 and 1e-30: the sums are in 64 bits."""
    announce("clip large and small values")
    for scale in (1e30, 1e-30):
        _check(_grads([5000, 70], seed=5, scale=scale, kinds="f"), 0.5 * scale)


def test_norm_only_and_zero():
    announce("clip norm only")
    g = _grads([5000, 70], seed=6)
    kept = [t.clone() for t in g]
    norm, _ = binding.clip_gradients(g, math.inf)
    assert abs(float(norm) - _block.clip(g, 1.0)[0]) <= 2 * _block.U32 * float(norm)
    assert all(torch.equal(a, b) for a, b in zip(g, kept))
    binding.clip_gradients(g, 0.0)
    assert not any(t.any() for t in g)


def test_refusals():
    g = _grads([100, 100])
    for bad, what in (([g[0], g[0]], "invalid"), ([g[0], g[0][50:]], "invalid"), ([], "no gradients"),
                      ([g[0].half()], "dtype"), ([g[0].cpu()], "no tensor given"), ([g[0], g[1].cpu()], "one GPU"),
                      ([torch.zeros((4, 4), device="cuda").T], "contiguous")):
        with pytest.raises(binding.MoELoRAError, match=what):
            binding.clip_gradients(bad, 1.0)
    for bad in (-1.0, float("nan")):
        with pytest.raises(binding.MoELoRAError, match="invalid"):
            binding.clip_gradients(g, bad)
    with pytest.raises(binding.MoELoRAError, match="tensors"):
        binding.clip_gradients(g, 1.0, out=g[:1])
    with pytest.raises(binding.MoELoRAError, match="invalid"):      # one tensor's output over another's input
        binding.clip_gradients([g[0], torch.zeros(100, device="cuda")], 1.0, out=[torch.zeros(100, device="cuda"), g[0]])
    with pytest.raises(binding.MoELoRAError, match="workspace"):
        binding.clip_gradients(g, 1.0, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_many_values():
    """More than 32 MB, whose results are written past the caches; the largest blocks."""
    for sizes in ([9_000_001, 3_000_003, 5], [17_000_001, 3_000_003, 5]):
        announce(f"clip {sizes}")
        _check(_grads(sizes, seed=8), 1.0)
        _check(_grads(sizes, seed=8), 1.0, in_place=True)
