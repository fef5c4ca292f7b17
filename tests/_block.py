"""Products with an epilogue, block norms and clipping in float64, from their
formulas (torch, on the tensors' device), with bounds on what fp32 sums and the
stated roundings may differ by.

Bounds: a bf16 rounding is off by at most U16 = 2^-8 of the value, an fp32 one by
U32 = 2^-24; a sum of n fp32 terms, in any order, by n 2 U32 sum |terms| (a step
may round by a whole unit in the matrix units)."""
import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24
TINY = 1e-30     # values below are 0 to every bound
ACTS = ("none", "relu", "gelu", "silu", "swiglu")
C = math.sqrt(2 / math.pi)


def act(name, z):
    """(value, slope) of an activation of one argument."""
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "gelu":
        u = C * (z + 0.044715 * z ** 3)
        t = torch.tanh(u)
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    return z, torch.ones_like(z)


def linear(x, w, name, bias=None, residual=None, fp32=False):
    """(out, bound, preact, its bound) of bf16 x [M, K], w [K, W]."""
    x, w = x.double(), w.double()
    K = x.shape[1]
    z, mag = x @ w, x.abs() @ w.abs()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    dz = (K + 2) * 2 * U32 * mag                       # the sum and the bias
    if name == "swiglu":
        N = w.shape[1] // 2
        g, u, dg, du = z[:, :N], z[:, N:], dz[:, :N], dz[:, N:]
        s, _ = act("silu", g)
        out = s * u
        # |silu'| < 1.1; the exponent's own rounding costs |g| units, 8 more operations one each
        off = 1.1 * dg * (u.abs() + du) + s.abs() * du + (g.abs() + 8) * 2 * U32 * out.abs()
    else:
        out, _ = act(name, z)
        off = 1.2 * dz + (z.abs() + 8) * 2 * U32 * out.abs()
        if name == "gelu":   # the exponent is cubic in z
            off = off + 4 * (z.abs() + 0.05 * z.abs() ** 3) * 2 * U32 * out.abs()
    if residual is not None:
        out = out + residual.double()
        off = off + U32 * out.abs() + U32 * residual.double().abs()
    return out, off + (U32 if fp32 else U16) * (out.abs() + off) + TINY, z, dz + U16 * (z.abs() + dz) + TINY


def linear_backward(x, w, d_out, name, preact=None):
    """{name: (value, bound)} of d_x, d_w, d_bias; dz is rounded to bf16 in the products."""
    x, w, d = x.double(), w.double(), d_out.double()
    rel = 0.0                      # of dz before its rounding, against `size`
    size = d.abs()
    if name == "swiglu":
        N = w.shape[1] // 2
        g, u = preact.double()[:, :N], preact.double()[:, N:]
        s, slope = act("silu", g)
        # the slope's two terms, and the exponent's rounding: |g| units
        size = torch.cat([d.abs() * u.abs() * (1.1 + g.abs() * 0.25) * (g.abs() + 8),
                          (d * s).abs() * (g.abs() + 8)], 1)
        d = torch.cat([d * u * slope, d * s], 1)
        rel = 2 * U32
    elif name != "none":
        z = preact.double()
        _, slope = act(name, z)
        cubic = z.abs() + (0.05 * z.abs() ** 3 if name == "gelu" else 0)
        size = d.abs() * (1.1 + z.abs() * (1 + z.abs()) * 0.5) * (4 * cubic + 8)
        # far out the slope's second term is 0 in fp32 and in the formula
        size = torch.where(cubic > 60, d.abs(), size)
        d = d * slope
        rel = 2 * U32
    off = rel * size
    M, W = d.shape
    part = off + U16 * (d.abs() + off)
    if name == "none" and d_out.dtype == torch.bfloat16:
        part = off                 # d_out enters as it is
    aw, ax = w.abs(), x.abs()
    d_x, d_w = d @ w.T, x.T @ d
    mag = d.abs() + part
    b_x = part @ aw.T + (W + 2) * 2 * U32 * (mag @ aw.T)
    b_w = ax.T @ part + (M + 2) * 2 * U32 * (ax.T @ mag)
    b_b = off.sum(0) + (M + 2) * U32 * (d.abs() + off).sum(0)
    return {"d_x": (d_x, b_x + U16 * (d_x.abs() + b_x) + TINY), "d_w": (d_w, b_w + U16 * (d_w.abs() + b_w) + TINY),
            "d_bias": (d.sum(0), b_b + TINY)}


def _rms(v, eps):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + eps)


def norm(x, y, w_post, w_pre, gate, eps, alpha, offset):
    """(new residual, bound, normed, bound); gate is [T, 1], [H] or None."""
    some = x if x is not None else y
    T, H = some.shape
    n = (H + 16) * U32              # of a root mean square: H terms of one sign, rsqrt, products
    b = torch.zeros((T, H), dtype=torch.float64, device=some.device)
    if y is not None:
        b = y.double()
        if w_post is not None:
            b = b * _rms(b, eps) * (offset + w_post.double())
        if gate is not None:
            b = b * gate.double()
    ax = torch.zeros_like(b) if x is None else alpha * x.double()
    # offset + w rounds against the larger of the two
    wide = 1.0 if w_post is None else 1 + (abs(offset) + w_post.double().abs()) / (
        (offset + w_post.double()).abs() + TINY)
    off = b.abs() * (n + 6 * U32 * wide) + 3 * U32 * (ax.abs() + b.abs())
    r = ax + b
    if w_pre is None:
        return r, off + U16 * (r.abs() + off) + TINY, None, None
    p = _rms(r, eps)
    w = offset + w_pre.double()
    z = r * p * w
    # p moves with the errors of r as their 2-norm does
    share = (off * off).sum(1, keepdim=True).sqrt() * p / math.sqrt(H)
    off_z = p * w.abs() * off + z.abs() * (share + n + 6 * U32) + p * r.abs() * 2 * U32 * (
        abs(offset) + w_pre.double().abs())
    return r, off + U16 * (r.abs() + off) + TINY, z, off_z + U16 * (z.abs() + off_z) + TINY


def norm_backward(r, y, w_post, w_pre, gate, d_r, d_z, eps, alpha, offset, per_token):
    """{name: (value, bound)} of the gradients; None where there is no input.  Each
    bound counts the roundings of the terms a value is made of, in magnitudes."""
    some = d_r if d_r is not None else d_z
    T, H = some.shape
    n = (H + 32) * 2 * U32
    zero = torch.zeros(some.shape, dtype=torch.float64, device=some.device)
    D = zero if d_r is None else d_r.double()
    mag = D.abs()
    out = {"residual": None, "branch": None, "post_weight": None, "pre_weight": None, "gate": None}
    if d_z is not None:
        r, dz = r.double(), d_z.double()
        p = _rms(r, eps)
        rh = r * p
        w = offset + w_pre.double()
        aw = abs(offset) + w_pre.double().abs()
        q = dz * w
        D = D + p * (q - rh * (q * rh).mean(1, keepdim=True))
        mag = mag + p * (dz.abs() * aw + rh.abs() * (dz.abs() * aw * rh.abs()).mean(1, keepdim=True))
        m = (dz * rh).abs()
        out["pre_weight"] = ((dz * rh).sum(0), (n + (T + 8) * U32) * m.sum(0) + TINY)
    off = 2 * n * mag                     # of D
    out["residual"] = (alpha * D, abs(alpha) * off * 2 + U16 * (alpha * D).abs() * (1 + 1e-3) + TINY)
    g = torch.ones((), dtype=torch.float64, device=some.device) if gate is None else gate.double()
    d, dm, do = g * D, g.abs() * mag, g.abs() * off
    if y is not None:
        yh, wp, awp = y.double(), torch.ones(H, dtype=torch.float64, device=some.device), 1.0
        s = torch.ones((T, 1), dtype=torch.float64, device=some.device)
        if w_post is not None:
            s = _rms(yh, eps)
            yh = yh * s
            wp, awp = offset + w_post.double(), abs(offset) + w_post.double().abs()
            out["post_weight"] = ((d * yh).sum(0),
                                  ((do + (n + (T + 8) * U32) * (d.abs() + do)) * yh.abs()).sum(0) + TINY)
        if gate is not None:
            b = yh * wp
            over = 1 if per_token else 0
            terms = (off + (n + (T + H) * U32) * (D.abs() + off)) * (yh * awp).abs()
            out["gate"] = ((D * b).sum(over), terms.sum(over) + TINY)
        h, hm = d * wp, dm * awp
        if w_post is not None:
            dy = s * (h - yh * (h * yh).mean(1, keepdim=True))
            ym = s * (hm + yh.abs() * (hm * yh.abs()).mean(1, keepdim=True))
        else:
            dy, ym = h, hm
        o = 4 * n * ym
        out["branch"] = (dy, o + U16 * (dy.abs() + o) + TINY)
    return out


def clip(gradients, max_norm):
    """(norm, factor, scaled gradients in float64)."""
    total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in gradients))
    f = min(1.0, max_norm / (total + 1e-6)) if math.isfinite(total) else 1.0
    return total, f, [g.double() * f for g in gradients]


def apart(got, want):
    """2-norm of the difference over that of the values: a worst case over thousands of
    terms hides a lost step of them, this does not.  A rounding to bf16 stays below U16,
    one of an operand as well (its errors have random signs)."""
    n = float(want.norm())
    return float((got.double() - want).norm()) / n if n else 0.0


def worst(got, want, bound):
    """Largest share of the bound that is used (NaN fails)."""
    d = (got.double() - want).abs() / bound
    return float(torch.nan_to_num(d, nan=float("inf")).max()) if d.numel() else 0.0
