"""The 4-bit products where a block runs several slab groups of its rows in
turn: the code ring, the staged activations, the accumulators and the LoRA
expand start over per group, and the last job may be shorter.  Every output row
against the definition in float64."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _w4
from tests._gpu import announce, bf16_to_np
from tests._w4 import W4Case
from tests.test_w4_launch import BLOCKS


def _product(x, w, scale, a, b, mapping, sums):
    """x W (+ its LoRA) per row, its error bound from that of x: fp32 sums of
    offset products (62 scale per weight, as in _w4.reference) and bf16 shrink
    outputs.  x, sums: (value, error); a, b: the expert's stacks by adapter."""
    v, dv = x
    y = v @ w
    dy = dv @ np.abs(w) + sums * ((np.abs(v) + dv) @ scale)
    for l in range(len(a) if a is not None else 0):
        r = mapping == l
        A, B = a[l].astype(np.float64), b[l].astype(np.float64)
        s = v[r] @ A.T
        ds = dv[r] @ np.abs(A).T + 2.0 ** -24 * v.shape[1] * ((np.abs(v[r]) + dv[r]) @ np.abs(A).T)
        y[r] += s @ B.T
        dy[r] += (ds + _w4.U * (np.abs(s) + ds)) @ np.abs(B).T
    return y, dy


def _reference(c, x):
    """(out, bound) as _w4.reference, a whole expert's rows at a time."""
    E_l, f32 = c.E_l or c.E, 2.0 ** -24
    ids, weights = _w4.route(c, x["logits"])
    out, bound = np.zeros((c.T, c.H)), np.zeros((c.T, c.H))
    for e in range(E_l):
        t, j = np.nonzero(ids == e + c.off)
        one = {n: {k: None if v is None else v[e:e + 1] for k, v in x[n].items()} for n in ("w13", "w2")}
        w13, w2 = (_w4.dequantise(one[n], c.group)[0] for n in ("w13", "w2"))
        s13, s2 = (62.0 * one[n]["scales"][0].astype(np.float64)[np.arange(K) // c.group]
                   for n, K in (("w13", c.H), ("w2", c.I)))
        m, v = x["mapping"][t], x["hidden"][t].astype(np.float64)
        h, dh = _product((v, np.zeros_like(v)), w13, s13, x["a_gu"][:, e] if c.rg else None, x["b_gu"][:, e],
                         m, f32 * (c.H + c.group))
        g, u, dg, du = h[:, :c.I], h[:, c.I:], dh[:, :c.I], dh[:, c.I:]
        sig = 1 / (1 + np.exp(-g))
        act = g * sig * u
        dact = 1.1 * np.abs(u) * dg + np.abs(g * sig) * du + 1.1 * dg * du
        dact = dact + (_w4.U + 16 * f32) * (np.abs(act) + dact)
        y, dy = _product((act, dact), w2, s2, x["a_dn"][:, e] if c.rd else None, x["b_dn"][:, e], m,
                         f32 * (c.I + c.group))
        wt = weights[t, j][:, None]
        out[t] += wt * y                       # a token has an expert once
        bound[t] += wt * (dy + f32 * 8 * c.k * np.abs(y))
    out, bound = out * c.scaling, bound * abs(c.scaling)
    return out, bound + _w4.U * (np.abs(out) + bound) + 1e-30


def test_reference_is_the_one_by_tokens():
    for c in (W4Case("a", 30, 192, 96, 5, 2, L=2, rg=8, rd=5, zeros=1, group=32, scaling=2.0),
              W4Case("b", 30, 64, 32, 8, 3, off=2, E_l=4, L=1, rg=0, rd=8, method=1)):
        x = _w4.inputs(c)
        (a, da), (b, db, _) = _reference(c, x), _w4.reference(c, x)
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-15)
        np.testing.assert_allclose(da, db, rtol=0.05)


@pytest.mark.gpu
@pytest.mark.parametrize("spec", BLOCKS, ids=lambda s: s["name"])
def test_blocks_of_several_slab_groups(spec):
    c = W4Case(**spec)
    announce(f"forward_w4 {c}")
    x = _w4.inputs(c)
    shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
    got = bf16_to_np(binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, **kw))
    torch.cuda.synchronize()
    ref, bound = _reference(c, x)
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), f"{(over > 0).sum()} of {over.size} outside, worst {over.max():.3e}"
