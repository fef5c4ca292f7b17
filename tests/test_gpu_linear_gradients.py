"""Gradients of products whose incoming gradients are infinite, zero beside huge
pre-activations, or fp32, against float64."""
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


# fp32 incoming gradients: as many bits of them as two bf16 values hold.  Half a step of the
# first is at most 2^-8 of the value, of the second at most 2^-8 of the first's error.
@pytest.mark.parametrize("act", _block.ACTS)
@pytest.mark.parametrize("M,K,N", [(1, 64, 128), (5, 512, 60), (65, 200, 17), (1000, 512, 128), (333, 416, 99),
                                   (300, 2048, 2056), (8192, 512, 128), (4100, 264, 130), (2500, 8, 1)])
def test_fp32_gradients_keep_their_bits(M, K, N, act):
    announce(f"linear_backward fp32 {M} {K} {N} {act}")
    shape, x, w, d, pre = _inputs(M, K, N, act, 23, True)
    got = binding.linear_backward(shape, x, w, d, preact=pre, bias_grad=True)
    exact = _block.linear_backward(x, w, d, act, pre)
    again = binding.linear_backward(shape, x.clone(), w, d, preact=pre, bias_grad=True)

    def right(name, t):
        value, _ = exact[name]
        assert _block.worst(t, *exact[name]) <= 1, name
        if t.numel() >= 64 and name != "d_bias":
            # one rounding of the result, which `once` is, and beside it 2^-16 for dz and
            # less than as much for fp32 sums and slopes of terms with random signs
            once = _block.apart(value.bfloat16(), value)
            assert _block.apart(t, value) <= once + 2.0 ** -14, name

    for name, t in got.items():
        right(name, t)
        assert torch.equal(t, again[name]), name
    # one gradient alone may be summed in other pieces
    right("d_x", binding.linear_backward(shape, x, w, d, preact=pre, w_grad=False)["d_x"])
    right("d_w", binding.linear_backward(shape, x, None, d, preact=pre, x_grad=False)["d_w"])
    inside = x.clone()          # in place: d_w is taken before d_x overwrites x
    over = binding.linear_backward(shape, inside, w, d, preact=pre, d_x=inside, bias_grad=True)
    for name, t in over.items():
        right(name, t)


def test_fp32_gradients_that_are_not_finite():
    """They stay in their rows and columns, and infinities stay infinities."""
    announce("linear_backward fp32 not finite")
    for M, K, N in ((40, 72, 17), (700, 264, 128)):
        shape, x, w, d, _ = _inputs(M, K, N, "none", 24, True)
        want = binding.linear_backward(shape, x, w, d, bias_grad=True)
        x[3], w[:, 5] = 1.0, 1.0
        base = binding.linear_backward(shape, x, w, d, bias_grad=True)
        d[3, 5] = float("inf")
        got = binding.linear_backward(shape, x, w, d, bias_grad=True)
        rows, cols = [i for i in range(M) if i != 3], [i for i in range(N) if i != 5]
        assert (got["d_x"][3] == float("inf")).all() and (got["d_w"][:, 5] == float("inf")).all()
        assert torch.equal(got["d_x"][rows], base["d_x"][rows]) and torch.equal(got["d_w"][:, cols], base["d_w"][:, cols])
        assert float(got["d_bias"][5]) == float("inf") and torch.isfinite(want["d_bias"]).all()
