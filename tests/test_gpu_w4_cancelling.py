"""The 4-bit products where their sums cancel: x (16 + code) and x (16 + zero
point) are summed apart, so weights of 0 and activations of one sign lose digits
that the definition does not.  The bound is the reference's, relative to the sum
of |x| scale (32 + code + zero point), with its largest value 62."""
import numpy as np
import pytest

from mixture_experts_layer_up_amd import binding
from tests import _w4
from tests._gpu import announce, bf16_to_np
from tests._w4 import W4Case
from tests.test_gpu_w4_blocks import _reference

pytestmark = pytest.mark.gpu

CASES = [
    W4Case("rows16", 40, 1088, 416, 8, 2, L=2, rg=8, rd=16, zeros=1, group=64),
    W4Case("rows16_group32", 3, 2048, 768, 4, 2, zeros=1, group=32),
    W4Case("rows32", 400, 320, 160, 2, 1, L=1, rg=8, rd=8, group=128),
    W4Case("rows64", 4100, 320, 160, 3, 1, zeros=1, group=64),
]


def _check(c, x):
    """(outputs, reference), the one within the bound of the other."""
    shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
    got = bf16_to_np(binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, **kw))
    ref, bound = _reference(c, x)
    assert (np.abs(got - ref) <= bound).all()
    return got, ref


@pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
def test_activations_of_one_sign(c):
    """A mean of 8 deviations: every group sum is about 8 group, its column sums
    mostly cancel."""
    announce(f"large mean {c}")
    x = _w4.inputs(c)
    x["hidden"] = _w4.bf16(x["hidden"] + np.where(np.arange(c.T) % 2, 8, -8)[:, None])
    for n in ("w13", "w2"):                     # keeps the layer's outputs of order 1
        x[n]["scales"] = _w4.bf16(x[n]["scales"] / 8)
    _check(c, x)


@pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
def test_large_activations_meet_weights_of_zero(c):
    """A few channels of 1000 deviations whose weights are all 0 (code = zero
    point): by definition they add nothing."""
    announce(f"zero weights {c}")
    x = _w4.inputs(c)
    loud = [1, c.H // 2, c.H - 2]
    q = x["w13"]
    z = q["zeros"] if q["zeros"] is not None else np.full(q["scales"].shape, 8, np.uint8)
    for k in loud:
        shift = 4 * (k & 1)
        q["codes"][:, k // 2] = (q["codes"][:, k // 2] & (0xf0 >> shift)) | (z[:, k // c.group] << shift)
    quiet = dict(x, hidden=x["hidden"].copy())
    quiet["hidden"][:, loud] = 0
    x["hidden"] = _w4.bf16(x["hidden"] * np.where(np.isin(np.arange(c.H), loud), 1000, 1))
    x["a_gu"][..., loud] = 0                    # the adapters do not see those channels either
    got, ref = _check(c, x)
    want, _ = _reference(c, quiet)
    np.testing.assert_allclose(ref, want, rtol=1e-9, atol=1e-9 * np.abs(want).max())
    # and leave less than the layer's bf16 roundings: a few 2^-24 of 31000 scale, against
    # 2^-8 of a sum of order sqrt(K) x 5 scale
    assert np.abs(got - ref).max() <= 8 * _w4.U * np.abs(ref).max()


@pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
def test_codes_equal_to_the_zero_point(c):
    """All down weights 0: the outputs are 0 within the bound."""
    announce(f"codes at the zero point {c}")
    x = _w4.inputs(c)
    q = x["w2"]
    z = q["zeros"] if q["zeros"] is not None else np.full(q["scales"].shape, 8, np.uint8)
    at = np.arange(0, c.I, 2) // c.group
    q["codes"][:] = z[:, at] | z[:, at] << 4
    x["mapping"][:] = -1
    assert (_check(c, x)[1] == 0).all()
