"""The 4-bit layer at the largest hidden and inter sizes, expert counts and top-k
that a shape may have, every output row against the definition in float64."""
import numpy as np
import pytest

from mixture_experts_layer_up_amd import binding
from tests import _w4
from tests._gpu import announce, bf16_to_np
from tests._w4 import W4Case
from tests.test_gpu_w4_blocks import _reference

pytestmark = pytest.mark.gpu

CASES = [
    W4Case("hidden_rows16", 5, 65536, 32, 2, 1, L=2, rg=8, rd=8, zeros=1, group=32),
    W4Case("hidden_rows16_odd", 9, 65472, 32, 2, 2, L=1, rg=12, rd=20, group=128),
    W4Case("hidden_rows32", 400, 65536, 32, 2, 1, L=2, rg=16, rd=8, group=64),
    W4Case("inter_rows16", 5, 64, 65536, 2, 1, L=2, rg=8, rd=8, zeros=1, group=64),
    W4Case("inter_rows16_odd", 9, 64, 65504, 2, 2, L=1, rg=20, rd=12, zeros=1, group=32),
    W4Case("inter_rows32", 400, 64, 65536, 2, 1, L=2, rg=8, rd=16, group=128),
    W4Case("inter_rows64", 4100, 64, 16384, 2, 1, zeros=1, group=64),
    W4Case("experts1024_top64", 3, 64, 32, 1024, 64, L=8, rg=8, rd=8, zeros=1, group=64),
    W4Case("experts1024_rows32", 340, 64, 32, 1024, 64, L=8, rg=8, rd=8, group=32),
    W4Case("experts1024_shard", 2000, 128, 64, 1024, 8, off=1000, E_l=24, L=64, rg=8, rd=4),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
def test_largest_sizes(c):
    announce(f"forward_w4 {c}")
    x = _w4.inputs(c)
    if max(c.H, c.I) > 10000:    # outputs of order 1 to 1000: sums of many thousand products
        for n in ("w13", "w2"):
            x[n]["scales"] = _w4.bf16(x[n]["scales"] / 8)
    shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
    got = bf16_to_np(binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, **kw))
    ref, bound = _reference(c, x)
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), f"{(over > 0).sum()} of {over.size} outside, worst {over.max():.3e}"
    # and near: a few bf16 roundings of the rows' 2-norms
    err = np.linalg.norm(got - ref, axis=1)
    assert (err <= 4 * _w4.U * np.linalg.norm(ref, axis=1)).all()
