"""moe_lora_block_norm and its gradients on the GPU against float64, within bounds
counted from the roundings (tests/_block.py)."""
import itertools

import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _block
from tests._gpu import announce

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _inputs(T, H, gate, seed, offset=0.0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    size = r(H).exp()
    d = {"x": (r(T, H) * size).bfloat16(), "y": (r(T, H) * size.flip(0)).bfloat16(),
         "w_post": (r(H) * 0.3 + 1 - offset).bfloat16(), "w_pre": (r(H) * 0.3 + 1 - offset).bfloat16(),
         "d_r": (r(T, H) * 0.1).bfloat16(), "d_z": (r(T, H) * 0.1).bfloat16(), "gate": None, "wide": None}
    if gate == "token":
        d["gate"] = r(T)
        d["wide"] = d["gate"][:, None]
    elif gate == "channel":
        d["gate"] = d["wide"] = r(H).bfloat16()
    return d


def _shape(T, H, gate, alpha=1.0, offset=0.0):
    return binding.NormShape(T, H, EPS, alpha, offset, binding.GATES.index(gate))


def _forward(T, H, gate="none", alpha=1.0, offset=0.0, post=True, pre=True, x=True, y=True, seed=1):
    announce(f"block_norm {T} {H} {gate} post={post} pre={pre} x={x} y={y}")
    d = _inputs(T, H, gate, seed, offset)
    x, y = d["x"] if x else None, d["y"] if y else None
    w_post, w_pre = d["w_post"] if post else None, d["w_pre"] if pre else None
    r, z = binding.block_norm(_shape(T, H, gate, alpha, offset), x, y, post_weight=w_post, pre_weight=w_pre,
                              gate=d["gate"])
    want_r, off_r, want_z, off_z = _block.norm(x, y, w_post, w_pre, d["wide"], EPS, alpha, offset)
    assert _block.worst(r, want_r, off_r) <= 1 and _block.apart(r, want_r) <= _block.U16
    assert (z is None) == (not pre)
    if pre:
        assert _block.worst(z, want_z, off_z) <= 1 and _block.apart(z, want_z) <= _block.U16
    return d, r, z


WIDTHS = [64, 128, 192, 256, 320, 512, 576, 1024, 1088, 1536, 2048, 2112, 2816, 3584, 4096, 5120, 6144, 7168, 8192,
          8256, 16384, 20480, 32768, 65536]


@pytest.mark.parametrize("H", WIDTHS)
def test_forward_widths(H):
    _forward(5, H, "channel", 0.5, 1.0)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 7, 333, 2049])
def test_forward_rows(T):
    _forward(T, 320, "token")
    _forward(T, 2048)


@pytest.mark.parametrize("gate,post,pre,x,y", [
    c for c in itertools.product(("none", "token", "channel"), (False, True), (False, True), (False, True),
                                 (False, True))
    if (c[3] or c[4]) and (c[4] or (not c[1] and c[0] == "none"))])
def test_forward_parts(gate, post, pre, x, y):
    for H in (192, 2048):
        _forward(9, H, gate, 0.7, 1.0, post, pre, x, y)


def test_forward_in_place_and_alone():
    """Outputs over the inputs, and one output alone: the same bits."""
    announce("block_norm in place")
    for H in (128, 2048, 16384):
        d, r, z = _forward(6, H, "channel")
        kw = dict(post_weight=d["w_post"], pre_weight=d["w_pre"], gate=d["gate"])
        sh = _shape(6, H, "channel")
        only, z2 = binding.block_norm(sh, d["x"], d["y"], residual_out=False, **kw)
        assert only is None and torch.equal(z2, z)
        x, y = d["x"].clone(), d["y"].clone()
        binding.block_norm(sh, x, y, new_residual=x, normed=y, **kw)
        assert torch.equal(x, r) and torch.equal(y, z)
        x, y = d["x"].clone(), d["y"].clone()
        binding.block_norm(sh, x, y, new_residual=y, normed=x, **kw)
        assert torch.equal(y, r) and torch.equal(x, z)


def test_rows_of_zeros_infinities_and_nan():
    """A row of zeros has norm eps; what is not finite stays in its row."""
    announce("block_norm special rows")
    for H in (256, 2048, 8192):
        d = _inputs(5, H, "none", 3)
        d["x"][0] = 0
        d["y"][0] = 0
        d["y"][2, 7] = float("inf")
        d["x"][3, H - 1] = float("nan")
        r, z = binding.block_norm(_shape(5, H, "none"), d["x"], d["y"], post_weight=d["w_post"],
                                  pre_weight=d["w_pre"])
        assert not r[0].any() and not z[0].any()
        rows = [1, 4]
        want_r, off_r, want_z, off_z = _block.norm(d["x"][rows], d["y"][rows], d["w_post"], d["w_pre"], None, EPS,
                                                   1.0, 0.0)
        assert _block.worst(r[rows], want_r, off_r) <= 1 and _block.worst(z[rows], want_z, off_z) <= 1
        assert torch.isnan(r[2]).any() and torch.isnan(z[2]).any() and torch.isnan(z[3]).all()
        r, z = binding.block_norm(_shape(5, H, "none"), d["x"], None, pre_weight=d["w_pre"])
        assert torch.equal(r[[0, 1, 2, 4]], d["x"][[0, 1, 2, 4]])


def _backward(T, H, gate="none", alpha=1.0, offset=0.0, post=True, d_r=True, d_z=True, y=True, seed=2):
    announce(f"block_norm_backward {T} {H} {gate} post={post} d_r={d_r} d_z={d_z} y={y}")
    d = _inputs(T, H, gate, seed, offset)
    y = d["y"] if y else None
    w_post, w_pre = d["w_post"] if post else None, d["w_pre"] if d_z else None
    d_r, d_z = d["d_r"] if d_r else None, d["d_z"] if d_z else None
    got = binding.block_norm_backward(_shape(T, H, gate, alpha, offset), d["x"] if d_z is not None else None, y,
                                      post_weight=w_post, pre_weight=w_pre, gate=d["gate"], d_residual=d_r,
                                      d_normed=d_z)
    want = _block.norm_backward(d["x"], y, w_post, w_pre, d["wide"], d_r, d_z, EPS, alpha, offset, gate == "token")
    for name in got:
        assert (got[name] is None) == (want[name] is None), name
        if got[name] is not None:
            v, off = want[name]
            share = _block.worst(got[name].view(v.shape), v, off)
            assert share <= 1, (name, share)
            near = _block.U16 if got[name].dtype == torch.bfloat16 else 1e-5
            assert _block.apart(got[name].view(v.shape), v) <= near, name
    return d, got


@pytest.mark.parametrize("H", WIDTHS)
def test_backward_widths(H):
    _backward(5, H, "channel", 0.5, 1.0)


@pytest.mark.parametrize("T", [1, 2, 17, 333, 5000])
def test_backward_rows(T):
    _backward(T, 320, "token")
    _backward(T, 2048, "channel")


@pytest.mark.parametrize("gate,post,d_r,d_z,y", [
    c for c in itertools.product(("none", "token", "channel"), (False, True), (False, True), (False, True),
                                 (False, True))
    if (c[2] or c[3]) and (c[4] or (not c[1] and c[0] == "none"))])
def test_backward_parts(gate, post, d_r, d_z, y):
    for H in (192, 2048):
        _backward(70, H, gate, 0.7, 1.0, post, d_r, d_z, y)


@pytest.mark.parametrize("gate", ["token", "channel"])
def test_backward_parts_alone_and_in_place(gate):
    announce("block_norm_backward parts alone")
    for T, H in ((300, 128), (300, 2048), (40, 1088), (30, 8256), (30, 16384)):
        d, every = _backward(T, H, gate)
        sh = _shape(T, H, gate)
        kw = dict(post_weight=d["w_post"], pre_weight=d["w_pre"], gate=d["gate"])
        for name in every:
            one = binding.block_norm_backward(sh, d["x"], d["y"], d_residual=d["d_r"], d_normed=d["d_z"],
                                              wanted=(name,), **kw)
            assert torch.equal(one[name], every[name])
            assert all(v is None for k, v in one.items() if k != name)
        for a, b in itertools.permutations(("x", "y", "d_r", "d_z"), 2):
            c = {k: d[k].clone() for k in ("x", "y", "d_r", "d_z")}
            got = binding.block_norm_backward(sh, c["x"], c["y"], d_residual=c["d_r"], d_normed=c["d_z"],
                                              out={"residual": c[a], "branch": c[b]}, **kw)
            assert all(torch.equal(got[k], every[k]) for k in every), (a, b)


def test_no_rows():
    announce("block_norm without rows")
    e = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    sh = _shape(0, 128, "channel")
    r, z = binding.block_norm(sh, e, e, post_weight=w, pre_weight=w, gate=w)
    assert r.shape == z.shape == (0, 128)
    got = binding.block_norm_backward(sh, e, e, post_weight=w, pre_weight=w, gate=w, d_residual=e, d_normed=e)
    assert all(not got[k].any() for k in ("post_weight", "pre_weight", "gate"))


def test_gradient_of_a_row_with_nan_stays_there():
    announce("block_norm_backward special rows")
    d = _inputs(6, 2048, "token", 5)
    d["d_z"][2, 9] = float("nan")
    got = binding.block_norm_backward(_shape(6, 2048, "token"), d["x"], d["y"], post_weight=d["w_post"],
                                      pre_weight=d["w_pre"], gate=d["gate"], d_residual=d["d_r"],
                                      d_normed=d["d_z"])
    rows = [0, 1, 3, 4, 5]
    assert torch.isfinite(got["residual"][rows]).all() and torch.isfinite(got["branch"][rows]).all()
    assert torch.isfinite(got["gate"][rows]).all() and torch.isnan(got["residual"][2]).all()
