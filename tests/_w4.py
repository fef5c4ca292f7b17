"""The layer with 4-bit expert weights in float64, token by token, with the
error that its bf16 roundings may leave, and seeded inputs for it.  Plain
numpy, written from the definition of the format and of the layer."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

from mixture_experts_layer_up_amd import binding
from mixture_experts_layer_up_amd.synth import bf16_bits_to_f32, f32_to_bf16_bits

U = torch.finfo(torch.bfloat16).eps / 2    # a bf16 rounding, relative


@dataclasses.dataclass(frozen=True)
class W4Case:
    name: str
    T: int
    H: int
    I: int
    E: int
    k: int
    off: int = 0
    E_l: int = 0          # 0: all
    L: int = 0
    rg: int = 0
    rd: int = 0
    group: int = 128
    zeros: int = 0
    method: int = 0
    scaling: float = 1.0
    shared: int = 0
    seed: int = 1

    def shape(self):
        return binding.Shape(self.T, self.H, self.I, self.E, self.k, self.off, self.E_l or self.E,
                             self.L, self.rg, self.rd, self.scaling, self.shared, self.method)

    def format(self):
        return binding.W4Format(self.group, self.zeros)


def bf16(a):
    """Rounded to bf16, as float32."""
    return bf16_bits_to_f32(f32_to_bf16_bits(np.asarray(a, np.float32)))


def weight(rng, E, K, N, group, zeros):
    """Codes over the whole range, scales of mixed size, plain layout (numpy)."""
    G = -(-K // group)
    return {"codes": rng.integers(0, 256, (E, K // 2, N)).astype(np.uint8),
            "scales": bf16(0.005 * np.exp(rng.normal(0, 0.5, (E, G, N)))),
            "zeros": rng.integers(0, 16, (E, G, N)).astype(np.uint8) if zeros else None}


def dequantise(q, group):
    codes = q["codes"]
    E, K2, N = codes.shape
    w = np.empty((E, 2 * K2, N))
    w[:, 0::2], w[:, 1::2] = codes & 15, codes >> 4
    g = np.arange(2 * K2) // group
    z = q["zeros"].astype(np.float64) if q["zeros"] is not None else np.full(q["scales"].shape, 8.0)
    return (w - z[:, g]) * q["scales"].astype(np.float64)[:, g]


def inputs(c: W4Case):
    rng = np.random.default_rng(c.seed)
    E_l, outer = c.E_l or c.E, 1 if c.shared else (c.E_l or c.E)
    return {
        "logits": rng.standard_normal((c.T, c.E)).astype(np.float32),
        "hidden": bf16(rng.standard_normal((c.T, c.H))),
        "w13": weight(rng, E_l, c.H, 2 * c.I, c.group, c.zeros),
        "w2": weight(rng, E_l, c.I, c.H, c.group, c.zeros),
        "mapping": rng.integers(-1, max(c.L, 1), c.T).astype(np.int32),
        "a_gu": bf16(0.1 * rng.standard_normal((c.L, outer, c.rg, c.H))),
        "b_gu": bf16(0.1 * rng.standard_normal((c.L, E_l, 2 * c.I, c.rg))),
        "a_dn": bf16(0.1 * rng.standard_normal((c.L, E_l, c.rd, c.I))),
        "b_dn": bf16(0.1 * rng.standard_normal((c.L, outer, c.H, c.rd))),
    }


def route(c: W4Case, logits):
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :c.k]
    v = logits.astype(np.float64)
    if not v.size:
        return ids, v[:, :c.k]
    top = np.exp(np.take_along_axis(v, ids, 1) - v.max(1, keepdims=True))
    every = np.exp(v - v.max(1, keepdims=True)).sum(1, keepdims=True)
    return ids, top / (every if c.method else top.sum(1, keepdims=True))


def reference(c: W4Case, x, ids=None, weights=None):
    """(out [T, H], its error bound, {(t, j): expert output}) in float64.

    The bound adds up, in absolute values, the roundings the operator states:
    shrink outputs, activations and the output to bf16 (U each), and fp32
    sums.  An fp32 sum of n products errs by at most n 2^-24 of the sum of the
    absolute products; with offsets up to (16 + 15) / 16 against |q - z|, and
    the products of the group sums, 2^-24 (K + group) (|x| |w|' ) with
    |w|' = s (16 + q + 16 + z) bounds it."""
    E_l = c.E_l or c.E
    if ids is None:
        ids, weights = route(c, x["logits"])
    w13, w2 = dequantise(x["w13"], c.group), dequantise(x["w2"], c.group)
    g13, g2 = np.arange(c.H) // c.group, np.arange(c.I) // c.group
    f32 = 2.0 ** -24
    out, bound = np.zeros((c.T, c.H)), np.zeros((c.T, c.H))
    slots = {}
    for t in range(c.T):
        h_t = x["hidden"][t].astype(np.float64)
        l = int(x["mapping"][t])
        for j in range(c.k):
            e = int(ids[t, j]) - c.off
            if not 0 <= e < E_l:
                continue
            o = 0 if c.shared else e
            s13 = 62.0 * x["w13"]["scales"][e].astype(np.float64)[g13]
            h = h_t @ w13[e]
            dh = f32 * (c.H + c.group) * (np.abs(h_t) @ s13)
            if 0 <= l < c.L and c.rg:
                s = x["a_gu"][l, o].astype(np.float64) @ h_t
                b = x["b_gu"][l, e].astype(np.float64)
                h = h + b @ s
                dh = dh + np.abs(b) @ (U * np.abs(s) + f32 * c.H *
                                       (np.abs(x["a_gu"][l, o]).astype(np.float64) @ np.abs(h_t)))
            g, u, dg, du = h[:c.I], h[c.I:], dh[:c.I], dh[c.I:]
            sig = 1 / (1 + np.exp(-g))
            act = g * sig * u
            # |silu'| <= 1.1; the hardware exponential and reciprocal: a few ulp
            dact = 1.1 * np.abs(u) * dg + np.abs(g * sig) * du + 1.1 * dg * du
            dact = dact + (U + 16 * f32) * (np.abs(act) + dact)
            s2 = 62.0 * x["w2"]["scales"][e].astype(np.float64)[g2]
            y = act @ w2[e]
            dy = dact @ np.abs(w2[e]) + f32 * (c.I + c.group) * ((np.abs(act) + dact) @ s2)
            if 0 <= l < c.L and c.rd:
                a = x["a_dn"][l, e].astype(np.float64)
                b = x["b_dn"][l, o].astype(np.float64)
                s = a @ act
                y = y + b @ s
                ds = np.abs(a) @ dact + f32 * c.I * (np.abs(a) @ np.abs(act))
                dy = dy + np.abs(b) @ (ds + U * (np.abs(s) + ds))
            slots[t, j] = y
            out[t] += weights[t, j] * y
            bound[t] += abs(weights[t, j]) * (dy + f32 * 8 * c.k * np.abs(y))
    out, bound = out * c.scaling, bound * abs(c.scaling)
    return out, bound + U * (np.abs(out) + bound) + 1e-30, slots


def device_layer(c: W4Case, x, device="cuda"):
    """The forward's keyword arguments and packed weights on the GPU."""
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    b = lambda a: dev(a.astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    q = [{"codes": dev(x[n]["codes"]), "scales": b(x[n]["scales"]),
          "zeros": dev(x[n]["zeros"]) if c.zeros else None} for n in ("w13", "w2")]
    shape, fmt = c.shape(), c.format()
    packed = binding.pack_weights_w4(shape, fmt, *q)
    a_gu, a_dn = binding.pack_lora_a(shape, b(x["a_gu"]), b(x["a_dn"]))
    kw = {"lora_a_gate_up": a_gu, "lora_b_gate_up": b(x["b_gu"]), "lora_a_down": a_dn,
          "lora_b_down": b(x["b_dn"]), "token_lora_mapping": dev(x["mapping"])}
    return shape, fmt, b(x["hidden"]), packed, kw, dev(x["logits"])
