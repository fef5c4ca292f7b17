"""moe_lora_linear and its gradients on the GPU against float64, within bounds
counted from the roundings (tests/_block.py)."""
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _block
from tests._gpu import announce

pytestmark = pytest.mark.gpu

GUARD = 64      # elements around every output that must stay as they are


def _guarded(shape, dtype):
    """A tensor between two guards, and a check that the guards are untouched."""
    n = 1
    for s in shape:
        n *= s
    flat = torch.full((n + 2 * GUARD,), 7.0, dtype=dtype, device="cuda")

    def intact():
        return bool((flat[:GUARD] == 7).all()) and bool((flat[GUARD + n:] == 7).all())

    return flat[GUARD:GUARD + n].view(shape), intact


def _make(M, K, N, act, seed, fp32=False):
    g = torch.Generator("cuda").manual_seed(seed)
    W = 2 * N if act == "swiglu" else N
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w = r(M, K).bfloat16(), (r(K, W) * (4 / K) ** 0.5).bfloat16()
    shape = binding.LinearShape(M, K, N, _block.ACTS.index(act), int(fp32))
    return shape, x, w, r(W), r(M, N), W


def _forward(M, K, N, act, fp32=False, bias=True, residual=True, preact=True, seed=1):
    announce(f"linear {M} {K} {N} {act} fp32={fp32}")
    shape, x, w, b, res, W = _make(M, K, N, act, seed, fp32)
    b = b if bias else None
    res = res.bfloat16() if residual else None
    out, out_ok = _guarded((M, N), torch.float32 if fp32 else torch.bfloat16)
    z, z_ok = _guarded((M, W), torch.bfloat16)
    z = z if preact else None
    got = binding.linear(shape, x, w, bias=b, residual=res, out=out, preact=z)
    torch.cuda.synchronize()
    assert got is out and out_ok() and z_ok()
    want, bound, pre, pre_bound = _block.linear(x, w, act, b, res, fp32)
    assert _block.worst(out, want, bound) <= 1
    if M * N >= 64:
        assert _block.apart(out, want) <= (1e-5 if fp32 else _block.U16)
    if preact:
        assert _block.worst(z, pre, pre_bound) <= 1


@pytest.mark.parametrize("act", _block.ACTS)
@pytest.mark.parametrize("M,K,N", [(1, 64, 128), (3, 2048, 96), (16, 40, 17), (17, 72, 130), (33, 128, 36),
                                   (64, 1000, 8), (65, 64, 128), (100, 416, 1085), (129, 8, 1),
                                   (256, 256, 256), (300, 328, 72), (700, 72, 545),
                                   (1111, 64, 260), (4500, 136, 12), (6000, 8, 3)])
def test_forward(M, K, N, act):
    _forward(M, K, N, act)


@pytest.mark.parametrize("M,K,N,act", [(5, 2048, 60, "none"), (64, 2048, 128, "none"), (700, 2048, 128, "none"),
                                       (129, 264, 33, "swiglu"), (1, 8, 1, "gelu"),
                                       (900, 264, 333, "swiglu"), (3000, 72, 60, "silu")])
def test_forward_fp32(M, K, N, act):
    _forward(M, K, N, act, fp32=True)


@pytest.mark.parametrize("M,K,N,act", [(2048, 512, 1024, "swiglu"), (3001, 264, 2056, "silu"),
                                       (2050, 64, 4096, "none"), (513, 8200, 264, "relu"),
                                       (1, 4096, 16384, "none"), (40, 512, 9000, "gelu")])
def test_forward_large(M, K, N, act):
    """Every tile shape, sums split and whole, rows of a few users over wide weights."""
    _forward(M, K, N, act, bias=False, residual=False, preact=False)
    _forward(M, K, N, act, seed=2)


# sizes that reach every tile with every way to store it (whole with an epilogue, whole
# swiglu pairs, split sums of one and of two projections), and every body for few rows
@pytest.mark.parametrize("M,K,N,act", [
    (20, 8, 2056, "swiglu"), (8193, 8, 500, "swiglu"), (6000, 8192, 500, "none"), (6000, 8192, 250, "swiglu"),
    (8193, 8, 250, "swiglu"), (4097, 4096, 264, "gelu"), (6000, 4096, 99, "swiglu"), (8193, 8, 250, "silu"),
    (3000, 8192, 99, "none"), (4097, 4096, 99, "swiglu"), (8193, 8, 8, "swiglu"), (20, 8192, 1, "swiglu"),
    (5, 64, 8208, "swiglu")])
def test_forward_every_body(M, K, N, act):
    _forward(M, K, N, act)


@pytest.mark.parametrize("M,N", [(5, 96), (300, 96), (2048, 100), (2048, 2048)])
def test_residual_in_place(M, N):
    announce(f"linear residual in place {M} {N}")
    shape, x, w, b, res, _ = _make(M, 128, N, "none", 3)
    res = res.bfloat16()
    want, bound, _, _ = _block.linear(x, w, "none", b, res)
    binding.linear(shape, x, w, bias=b, residual=res, out=res)
    assert _block.worst(res, want, bound) <= 1


@pytest.mark.parametrize("M", [20, 200, 1000])
def test_unaligned_outputs(M):
    """Outputs, residual and bias one element off any boundary."""
    announce(f"linear unaligned {M}")
    K, N = 64, 136
    shape, x, w, b, res, _ = _make(M, K, N, "silu", 4)
    buf = torch.zeros(M * N + 1, dtype=torch.bfloat16, device="cuda")
    r1 = torch.zeros(M * N + 1, dtype=torch.bfloat16, device="cuda")
    r1[1:] = res.bfloat16().view(-1)
    b1 = torch.zeros(N + 1, device="cuda")
    b1[1:] = b
    out = buf[1:].view(M, N)
    binding.linear(shape, x, w, bias=b1[1:], residual=r1[1:].view(M, N), out=out)
    want, bound, _, _ = _block.linear(x, w, "silu", b, res.bfloat16())
    assert _block.worst(out, want, bound) <= 1 and float(buf[0]) == 0


def test_non_finite_values_stay_in_their_rows_and_columns():
    """An infinity in a row of x or a column of w reaches no other row or column, also in tails."""
    for M, K, N in ((20, 72, 100), (200, 72, 100), (300, 200, 300), (2000, 72, 100), (2000, 200, 304)):
        announce(f"linear non-finite {M} {K} {N}")
        shape, x, w, _, _, _ = _make(M, K, N, "none", 5)
        want, bound, _, _ = _block.linear(x, w, "none")
        x[M // 2, 3], x[M - 1, K - 1] = float("inf"), float("nan")
        w[K - 1, N - 1], w[0, 5] = float("-inf"), float("nan")
        out = binding.linear(shape, x, w)
        rows = [m for m in range(M) if m not in (M // 2, M - 1)]
        cols = [n for n in range(N) if n not in (N - 1, 5)]
        assert _block.worst(out[rows][:, cols], want[rows][:, cols], bound[rows][:, cols]) <= 1
        assert not torch.isfinite(out[M // 2]).any() and torch.isnan(out[M - 1]).all()
        assert torch.isnan(out[:, 5]).all() and not torch.isfinite(out[:, N - 1]).any()


def test_neighbours_are_not_read_into_the_product():
    """NaN around x and w (the next rows of a larger buffer) never enters."""
    for M, K, N in ((3, 40, 24), (70, 72, 40), (300, 136, 264), (2100, 136, 265), (2100, 72, 1040)):
        announce(f"linear neighbours {M} {K} {N}")
        shape, x, w, _, _, _ = _make(M, K, N, "none", 6)
        bx = torch.full((M + 40, K), float("nan"), dtype=torch.bfloat16, device="cuda")
        bw = torch.full((K + 64, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        bx[:M], bw[:K] = x, w
        want, bound, _, _ = _block.linear(x, w, "none")
        assert _block.worst(binding.linear(shape, bx[:M], bw[:K]), want, bound) <= 1


def _backward(M, K, N, act, fp32=False, bias=True, seed=11):
    announce(f"linear_backward {M} {K} {N} {act} fp32={fp32}")
    shape, x, w, _, d, W = _make(M, K, N, act, seed, fp32)
    d = d * 0.01 if fp32 else (d * 0.01).bfloat16()
    g = torch.Generator("cuda").manual_seed(seed + 100)
    pre = (torch.randn((M, W), generator=g, device="cuda") * 2).bfloat16() if act != "none" else None
    d_x, x_ok = _guarded((M, K), torch.bfloat16)
    d_w, w_ok = _guarded((K, W), torch.bfloat16)
    d_b, b_ok = _guarded((W,), torch.float32)
    got = binding.linear_backward(shape, x, w, d, preact=pre, d_x=d_x, d_w=d_w, d_bias=d_b, bias_grad=bias)
    torch.cuda.synchronize()
    assert x_ok() and w_ok() and b_ok()
    want = _block.linear_backward(x, w, d, act, pre)
    for name, t in got.items():
        if t is None:
            assert name == "d_bias" and not bias
            continue
        share = _block.worst(t, *want[name])
        assert share <= 1, (name, share)
        if t.numel() >= 64:
            assert _block.apart(t, want[name][0]) <= (1e-5 if name == "d_bias" else 2 * _block.U16), name


@pytest.mark.parametrize("act", _block.ACTS)
@pytest.mark.parametrize("M,K,N", [(1, 64, 128), (3, 200, 17), (64, 128, 8), (100, 72, 1), (130, 264, 260),
                                   (333, 416, 99)])
def test_backward(M, K, N, act):
    _backward(M, K, N, act)


@pytest.mark.parametrize("M,K,N,act,fp32,bias", [(5, 512, 60, "none", True, True), (1000, 512, 128, "none", True, True),
                                                 (4100, 512, 256, "swiglu", False, False),
                                                 (4096, 1024, 1024, "none", False, True),
                                                 (300, 2048, 2056, "gelu", True, False),
                                                 (2048, 4104, 64, "none", False, False)])
def test_backward_large(M, K, N, act, fp32, bias):
    _backward(M, K, N, act, fp32, bias)


# the same for the gradients: one launch for both or one each, whole or split, plain or padded
@pytest.mark.parametrize("M,K,N,act", [
    (1000, 8192, 777, "none"), (8193, 1024, 777, "swiglu"), (1000, 8192, 1024, "none"), (500, 8192, 500, "relu"),
    (500, 8192, 512, "none"), (257, 8192, 99, "swiglu"), (6000, 1024, 99, "silu"), (257, 8192, 128, "swiglu"),
    (20, 8192, 1030, "none"), (20, 2048, 2056, "swiglu"), (20, 1024, 3001, "swiglu"), (6000, 4096, 264, "none"),
    (20, 1024, 2056, "swiglu"), (20, 512, 3001, "swiglu"), (6000, 8192, 99, "swiglu"), (20, 512, 2056, "swiglu"),
    (20, 8, 1030, "swiglu"), (3000, 2048, 1, "none"), (2049, 2048, 4096, "swiglu"), (8193, 1024, 1, "gelu"),
    (3000, 512, 4096, "swiglu"), (257, 2048, 3001, "swiglu"), (20, 8, 2056, "none"), (20, 8192, 500, "swiglu")])
def test_backward_every_body(M, K, N, act):
    _backward(M, K, N, act)


def test_backward_extreme_preactivations():
    """Slopes far out are 0 or 1, never NaN: preactivations up to the type's range, zeros of both signs."""
    for act in ("relu", "gelu", "silu", "swiglu"):
        announce(f"linear_backward extreme {act}")
        shape, x, w, _, d, W = _make(40, 64, 24, act, 12)
        d = d.bfloat16()
        z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20, -20, 90, -90, 1e4, -1e4, 3e38, -3e38], device="cuda")
        pre = z[torch.arange(40 * W, device="cuda") % 12].view(40, W).bfloat16()
        if act == "swiglu":     # dz holds silu(gate): within the range of its sums
            pre = pre.clamp(-1e4, 1e4)
            pre[:, 24:] = 1.5
        got = binding.linear_backward(shape, x, w, d, preact=pre, bias_grad=True)
        want = _block.linear_backward(x, w, d, act, pre)
        for name, t in got.items():
            assert _block.worst(t, *want[name]) <= 1, (act, name)


def test_parts_alone_are_the_same_bits():
    announce("linear_backward parts")
    shape, x, w, _, d, W = _make(300, 136, 96, "silu", 13)
    d = d.bfloat16()
    pre = torch.randn((300, W), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    every = binding.linear_backward(shape, x, w, d, preact=pre, bias_grad=True)
    for name, kw in (("d_x", dict(w_grad=False)), ("d_w", dict(x_grad=False)),
                     ("d_bias", dict(x_grad=False, w_grad=False, bias_grad=True))):
        one = binding.linear_backward(shape, None if name != "d_w" else x, w if name == "d_x" else None, d,
                                      preact=pre, **kw)
        assert torch.equal(one[name], every[name])
        assert all(v is None for k, v in one.items() if k != name)
    again = binding.linear_backward(shape, x, w, d, preact=pre, bias_grad=True, d_x=x)   # in place
    assert again["d_x"] is x and all(torch.equal(again[k], every[k]) for k in every)


def test_no_rows():
    announce("linear without rows")
    shape = binding.LinearShape(0, 64, 24, 0, 0)
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((64, 24), dtype=torch.bfloat16, device="cuda")
    assert binding.linear(shape, empty, w).shape == (0, 24)
    d = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    got = binding.linear_backward(shape, empty, w, d, bias_grad=True)
    assert got["d_x"].shape == (0, 64) and not got["d_w"].any() and not got["d_bias"].any()


def test_runs_are_the_same_bits():
    for M, K, N in ((30, 512, 96), (200, 2048, 128), (2048, 512, 1024)):
        announce(f"linear repeat {M} {K} {N}")
        shape, x, w, b, res, _ = _make(M, K, N, "gelu", 14)
        first = binding.linear(shape, x, w, bias=b)
        assert all(torch.equal(binding.linear(shape, x, w, bias=b), first) for _ in range(3))
