"""The float64 gradients that the GPU tests compare with, against central
differences of the float64 forward formulas."""
import pytest
import torch

from tests import _block

H = 1e-5     # differences are off by about H^2 times a third derivative, and 1e-16 / H


def _differences(f, at, grad):
    """sum(grad * f) by each element of `at`."""
    out = torch.zeros_like(at)
    flat, o = at.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + H
        up = float((grad * f()).sum())
        flat[i] = keep - H
        down = float((grad * f()).sum())
        flat[i] = keep
        o[i] = (up - down) / (2 * H)
    return out


def _close(a, b):
    assert (a - b).abs().max() <= 1e-7 * (1 + b.abs().max())


@pytest.mark.parametrize("name", _block.ACTS)
def test_linear_gradients(name):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    M, K, N = 3, 8, 2
    W = 2 * N if name == "swiglu" else N
    x, w, b, d = r(M, K), r(K, W), r(W), r(M, N)
    pre = x @ w + b
    got = _block.linear_backward(x, w, d, name, pre)
    f = lambda: _block.linear(x, w, name, b)[0]  # noqa: E731
    _close(got["d_x"][0], _differences(f, x, d))
    _close(got["d_w"][0], _differences(f, w, d))
    _close(got["d_bias"][0], _differences(f, b, d))


@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("post", [False, True])
def test_norm_gradients(gate, post):
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    T, C = 3, 5
    x, y, wp, wq, d_r, d_z = r(T, C), r(T, C), r(C), r(C), r(T, C), r(T, C)
    gt = {"none": None, "token": r(T, 1), "channel": r(C)}[gate]
    eps, alpha, offset = 1e-3, 0.7, 1.0
    w_post = wp if post else None
    new = _block.norm(x, y, w_post, wq, gt, eps, alpha, offset)[0]
    got = _block.norm_backward(new, y, w_post, wq, gt, d_r, d_z, eps, alpha, offset, gate == "token")

    def both():
        a, _, z, _ = _block.norm(x, y, w_post, wq, gt, eps, alpha, offset)
        return torch.cat([a, z])

    d = torch.cat([d_r, d_z])
    _close(got["residual"][0], _differences(both, x, d))
    _close(got["branch"][0], _differences(both, y, d))
    _close(got["pre_weight"][0], _differences(both, wq, d))
    if post:
        _close(got["post_weight"][0], _differences(both, wp, d))
    if gt is not None:
        _close(got["gate"][0].view(gt.shape), _differences(both, gt, d))
