"""Products, norms and clipping of more than 2^31 values: offsets pass 32 bits.  Sampled
rows, and all columns' sums, against float64."""
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _block
from tests._gpu import announce

pytestmark = pytest.mark.gpu


def _fill(shape, seed, sigma=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, sigma, generator=g)


def _rows(M):
    return torch.tensor([0, 1, M // 3, (1 << 31) // 2056, M - 300, M - 2, M - 1], device="cuda").clamp(0, M - 1)


def test_product_with_a_large_output():
    M, K, N = (1 << 20) + 3, 64, 2056
    announce(f"linear {M} {K} {N}")
    sh = binding.LinearShape(M, K, N, 3, 0)
    x, w, res = _fill((M, K), 1), _fill((K, N), 2, 0.2), _fill((M, N), 3)
    pre = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    assert M * N > 1 << 31
    out = binding.linear(sh, x, w, residual=res, preact=pre)
    r = _rows(M)
    want, bound, z, off = _block.linear(x[r], w, "silu", None, res[r])
    assert _block.worst(out[r], want, bound) <= 1 and _block.worst(pre[r], z, off) <= 1


def test_gradients_of_a_large_input():
    M, K, N = (1 << 19) + 5, 4104, 8
    announce(f"linear_backward {M} {K} {N}")
    assert M * K > 1 << 31
    sh = binding.LinearShape(M, K, N, 0, 0)
    x, w, d = _fill((M, K), 4), _fill((K, N), 5, 0.2), _fill((M, N), 6)
    got = binding.linear_backward(sh, x, w, d, bias_grad=True)
    r = _rows(M)
    want, bound = _block.linear_backward(x[r], w, d[r], "none")["d_x"]
    assert _block.worst(got["d_x"][r], want, bound) <= 1
    exact = torch.zeros((K, N), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(exact)
    for part in range(0, M, 1 << 16):
        a, b = x[part:part + (1 << 16)].double(), d[part:part + (1 << 16)].double()
        exact += a.T @ b
        size += a.abs().T @ b.abs()
    # fp32 sums of M terms in any order, one bf16 rounding
    bound = M * 2 * _block.U32 * size
    assert _block.worst(got["d_w"], exact, bound + _block.U16 * (exact.abs() + bound)) <= 1
    # and as sums of random signs should be: a lost or repeated part of the rows would show
    assert float((got["d_w"].double() - exact).norm() / exact.norm()) < 2 * _block.U16
    total, mags = d.double().sum(0), d.double().abs().sum(0)
    assert _block.worst(got["d_bias"], total, M * 2 * _block.U32 * mags) <= 1
    assert float((got["d_bias"].double() - total).norm() / total.norm()) < 1e-4


def test_norms_of_a_large_batch():
    T, H = 525_001, 4096
    announce(f"block_norm {T} {H}")
    assert T * H > 1 << 31
    sh = binding.NormShape(T, H, 1e-6, 0.5, 0.0, 1)
    x, y = _fill((T, H), 7), _fill((T, H), 8)
    wp, wq = _fill((H,), 9), _fill((H,), 10)
    gate = torch.rand(T, generator=torch.Generator("cuda").manual_seed(11), device="cuda")
    r, z = binding.block_norm(sh, x, y, post_weight=wp, pre_weight=wq, gate=gate)
    at = _rows(T)
    want_r, off_r, want_z, off_z = _block.norm(x[at], y[at], wp, wq, gate[at][:, None], 1e-6, 0.5, 0.0)
    assert _block.worst(r[at], want_r, off_r) <= 1 and _block.worst(z[at], want_z, off_z) <= 1
    got = binding.block_norm_backward(sh, r, y, post_weight=wp, pre_weight=wq, gate=gate, d_residual=x, d_normed=z,
                                      out={"residual": x})
    # x was the gradient d_residual and now holds the residual's; the rows' inputs are drawn again
    before = _fill((T, H), 7)
    want = _block.norm_backward(r[at], y[at], wp, wq, gate[at][:, None], before[at], z[at], 1e-6, 0.5, 0.0, True)
    for name in ("residual", "branch", "gate"):
        v, off = want[name]
        assert _block.worst(got[name][at].view(v.shape), v, off) <= 1, name
    sums = torch.zeros(H, dtype=torch.float64, device="cuda")
    for part in range(0, T, 1 << 16):
        rr, dz = r[part:part + (1 << 16)].double(), z[part:part + (1 << 16)].double()
        sums += (dz * rr * torch.rsqrt((rr * rr).mean(1, keepdim=True) + 1e-6)).sum(0)
    assert float((got["pre_weight"].double() - sums).norm() / sums.norm()) < 1e-4


def test_clipping_a_large_tensor():
    n = (1 << 31) + 77
    announce(f"clip {n}")
    big, small = _fill((n,), 12, 0.01), _fill((1000,), 13)
    at = torch.tensor([0, 5, (1 << 31) - 1, 1 << 31, n - 1], device="cuda")
    kept = big[at].double()
    total = 0.0
    for part in range(0, n, 1 << 27):
        total += float((big[part:part + (1 << 27)].double() ** 2).sum())
    total = (total + float((small.double() ** 2).sum())) ** 0.5
    norm, _ = binding.clip_gradients([big, small], 1.0)
    assert abs(float(norm) - total) <= 1e-6 * total
    want = kept / (total + 1e-6)
    assert _block.worst(big[at], want, _block.U16 * want.abs() * 1.01 + 1e-30) <= 1
