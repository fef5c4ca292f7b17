"""Gradients of products whose incoming gradients are infinite, NaN, or zero beside huge
pre-activations."""
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _block
from tests._gpu import announce

pytestmark = pytest.mark.gpu


def _inputs(M, K, N, act, seed, fp32):
    g = torch.Generator("cuda").manual_seed(seed)
    W = 2 * N if act == "swiglu" else N
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w, d = r(M, K).bfloat16(), (r(K, W) * (4 / K) ** 0.5).bfloat16(), r(M, N) * 0.01
    pre = None if act == "none" else (2 * r(M, W)).bfloat16()
    return binding.LinearShape(M, K, N, _block.ACTS.index(act), int(fp32)), x, w, d if fp32 else d.bfloat16(), pre


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("M,K,N", [(7, 64, 24), (40, 72, 17), (300, 136, 264), (2100, 64, 1030)])
def test_relu_takes_nothing_from_units_that_are_off(M, K, N, fp32):
    """Where z <= 0 the gradient is 0, whatever comes in: infinities and NaN there are as zeros."""
    announce(f"linear_backward relu {M} {K} {N} fp32={fp32}")
    shape, x, w, d, pre = _inputs(M, K, N, "relu", 21, fp32)
    pre[0, 0], pre[M - 1, N - 1] = 0.0, -0.0
    off = pre.float() <= 0
    clean = torch.where(off, torch.zeros_like(d), d)
    want = binding.linear_backward(shape, x, w, clean, preact=pre, bias_grad=True)
    for bad in (float("inf"), float("-inf"), float("nan")):
        spoilt = torch.where(off, torch.full_like(d, bad), d)
        got = binding.linear_backward(shape, x, w, spoilt, preact=pre, bias_grad=True)
        for name, t in got.items():
            assert torch.equal(t, want[name]), (bad, name)
    # and a unit that is on passes an infinity through, in its row and column only
    m, n = [int(v) for v in (~off).nonzero()[0]]
    clean[m, n] = float("inf")
    got = binding.linear_backward(shape, x, w, clean, preact=pre, bias_grad=True)
    rows, cols = [i for i in range(M) if i != m], [i for i in range(N) if i != n]
    assert not torch.isfinite(got["d_x"][m]).any() and torch.equal(got["d_x"][rows], want["d_x"][rows])
    assert not torch.isfinite(got["d_w"][:, n]).any() and torch.equal(got["d_w"][:, cols], want["d_w"][:, cols])
    assert torch.isinf(got["d_bias"][n]) and torch.equal(got["d_bias"][cols], want["d_bias"][cols])


@pytest.mark.parametrize("N", [24, 17])
def test_swiglu_up_values_at_the_end_of_the_range(N):
    """up slope(gate) alone may pass the range, the gradient with it does not; rows of zero
    gradients add nothing beside any finite pre-activation."""
    announce(f"linear_backward swiglu large up {N}")
    M, K = 40, 64
    shape, x, w, d, pre = _inputs(M, K, N, "swiglu", 22, False)
    top = torch.finfo(torch.bfloat16).max
    pre[:, :N], pre[:, N:] = 2.4, top           # the slope of silu is 1.0998 at 2.4
    d[::2] = 0
    d[1::2] = (d[1::2].float() * 1e-35).bfloat16()
    got = binding.linear_backward(shape, x, w, d, preact=pre, bias_grad=True)
    want = _block.linear_backward(x, w, d, "swiglu", pre)
    for name, t in got.items():
        assert _block.worst(t, *want[name]) <= 1, name
    assert not got["d_x"][::2].any()
