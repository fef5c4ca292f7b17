"""Workloads of what stands around the routed layer in a block, serving and training.

Five operators, each with its plain form in elementary torch operations:

``linear``               product with bias, activation and residual (router logits, shared expert)
``linear_backward``      its gradients of input, weight and bias
``block_norm``           norm after the layer, gate, residual sum and the next norm in one
``block_norm_backward``  its gradients
``clip_gradients``       global norm over many gradients, and the clipped gradients

``own`` selects the framework's calls; otherwise the plain forms run.
"""
import math

import torch

own = False

DEV = "cuda"
ACTIVATIONS = ("none", "relu", "gelu", "silu", "swiglu")
GATES = ("none", "token", "channel")


# ---------------------------------------------------------------- the cases

def _linear(name, M, K, N, act="none", fp32=False, bias=False, residual=False):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "act": act, "fp32": fp32, "bias": bias,
            "residual": residual}


def _grad(name, M, K, N, act="none", fp32=False, bias=False):
    return {"name": name, "op": "linear_backward", "M": M, "K": K, "N": N, "act": act, "fp32": fp32,
            "bias": bias}


def _norm(name, op, T, H, gate, post=True, pre=True, scale=1.0, offset=0.0):
    return {"name": name, "op": op, "T": T, "H": H, "gate": gate, "post": post, "pre": pre, "scale": scale,
            "offset": offset}


def listed():
    return [
        # a shared expert's first product for one user's next token: latency
        _linear("linear one token", 1, 2048, 768, "swiglu"),
        # a decode batch's router logits, in the type that routing takes
        _linear("linear router 64", 64, 2048, 128, fp32=True, bias=True),
        # a training micro-batch through a wide shared expert: the matrix units
        _linear("linear shared 8192", 8192, 2048, 2048, "swiglu"),
        # sizes that fill no tile, rows of the weight that are not aligned, every part of the epilogue
        _linear("linear odd", 333, 416, 1085, "gelu", bias=True, residual=True),
        # a micro-batch's router: gradients of fp32 logits, few columns
        _grad("linear grad router", 8192, 2048, 128, fp32=True, bias=True),
        # the shared expert's first product in training: both products and the activation's gradient
        _grad("linear grad shared", 8192, 2048, 768, "swiglu"),
        # one token's residual sum between two norms, and a micro-batch's
        _norm("norm one token", "block_norm", 1, 2048, "none"),
        _norm("norm 8192", "block_norm", 8192, 2048, "channel", scale=0.5),
        # its gradients, with both norms' weights and the gate; and sizes that fill nothing
        _norm("norm grad 8192", "block_norm_backward", 8192, 2048, "channel", scale=0.5),
        _norm("norm grad odd", "block_norm_backward", 333, 1088, "token", offset=1.0),
        # a router's and two norms' gradients
        {"name": "clip few", "op": "clip_gradients", "tensors": 5, "largest": 2048 * 128, "bf16": 0.2, "clips": True},
        # the adapters of many layers: small tensors, some large ones
        {"name": "clip many", "op": "clip_gradients", "tensors": 60, "largest": 2048 * 2048, "bf16": 0.5,
         "clips": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "linear_backward", "block_norm",
                     "block_norm_backward", "clip_gradients"])
    if op == "linear":
        c = _linear("", _log(rng, 1, 8192), 8 * rng.randint(8, 256), _log(rng, 1, 2048), rng.choice(ACTIVATIONS),
                    rng.random() < 0.3, rng.random() < 0.5, rng.random() < 0.4)
    elif op == "linear_backward":
        c = _grad("", _log(rng, 1, 8192), 8 * rng.randint(8, 256), _log(rng, 1, 1024), rng.choice(ACTIVATIONS),
                  rng.random() < 0.3, rng.random() < 0.5)
    elif op == "clip_gradients":
        c = {"op": op, "tensors": _log(rng, 1, 60), "largest": _log(rng, 64, 2048 * 2048),
             "bf16": rng.choice([0.0, 0.5, 1.0]), "clips": rng.random() < 0.7}
    else:
        c = _norm("", op, _log(rng, 1, 8192), 64 * rng.randint(1, 40), rng.choice(GATES), rng.random() < 0.7,
                  rng.random() < 0.8, rng.choice([1.0, 0.5]), rng.choice([0.0, 1.0]))
    c.pop("name", None)
    return c


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _bf16(g, sigma, *shape):
    return (_randn(g, *shape) * sigma).to(torch.bfloat16)


def _width(c):
    return 2 * c["N"] if c["act"] == "swiglu" else c["N"]


def _sizes(c):
    """Elements of each gradient: from a few to the largest, spread over the logarithm, the first the largest."""
    n = c["tensors"]
    return [max(1, int(c["largest"] ** (1 - 0.6 * i / n))) for i in range(n)]


def _count_bf16(c):
    return int(round(c["bf16"] * c["tensors"]))


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] in ("linear", "linear_backward"):
        M, K, N, W = c["M"], c["K"], c["N"], _width(c)
        s["x"], s["w"] = _bf16(g, 1.0, M, K), _bf16(g, 0.02, K, W)
        s["bias"] = _randn(g, W) * 0.1 if c["bias"] else None
        if c["op"] == "linear":
            s["residual"] = _bf16(g, 1.0, M, N) if c["residual"] else None
        else:
            d = _randn(g, M, N) * 0.01
            s["d_out"] = d if c["fp32"] else d.to(torch.bfloat16)
            z = (s["x"] @ s["w"]).float()  # a program holds these from its forward pass
            z = z if s["bias"] is None else z + s["bias"]
            s["preact"] = z.to(torch.bfloat16) if c["act"] != "none" else None
        if own:
            from mixture_experts_layer_up_amd import binding
            sh = s["shape"] = binding.LinearShape(M, K, N, ACTIVATIONS.index(c["act"]), int(c["fp32"]))
            need = (binding.linear_workspace_size if c["op"] == "linear" else
                    binding.linear_backward_workspace_size)(sh)
            s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
        return s
    if c["op"] == "clip_gradients":
        few = _count_bf16(c)
        s["grads"] = [_randn(g, n) * (0.01 if i % 3 else 0.1) for i, n in enumerate(_sizes(c))]
        s["grads"] = [x.to(torch.bfloat16) if i >= c["tensors"] - few else x for i, x in enumerate(s["grads"])]
        s["out"] = [torch.zeros_like(x) for x in s["grads"]]
        s["max_norm"] = 0.5 if c["clips"] else 1e4
        if own:
            from mixture_experts_layer_up_amd import binding
            s["workspace"] = torch.empty(max(1, binding.clip_workspace_size(s["grads"])), dtype=torch.uint8,
                                         device=DEV)
        return s
    T, H = c["T"], c["H"]
    channel = _randn(g, H).exp()  # channels differ in size, as a block's do
    s["x"] = (_randn(g, T, H) * channel).to(torch.bfloat16)
    s["y"] = (_randn(g, T, H) * channel.flip(0)).to(torch.bfloat16)
    s["w_post"] = (_randn(g, H) * 0.2 + 1 - c["offset"]).to(torch.bfloat16) if c["post"] else None
    s["w_pre"] = (_randn(g, H) * 0.2 + 1 - c["offset"]).to(torch.bfloat16) if c["pre"] else None
    s["gate"] = {"none": lambda: None, "token": lambda: torch.rand(T, generator=g, device=DEV),
                 "channel": lambda: _bf16(g, 0.5, H)}[c["gate"]]()
    if c["op"] == "block_norm_backward":  # the residual stream as the forward pass left it
        s["r"] = _plain_norm(s)["residual"]
        s["d_r"] = _bf16(g, 0.01, T, H)
        s["d_z"] = _bf16(g, 0.01, T, H) if c["pre"] else None
    if own:
        from mixture_experts_layer_up_amd import binding
        sh = s["shape"] = binding.NormShape(T, H, 1e-6, c["scale"], c["offset"], GATES.index(c["gate"]))
        if c["op"] == "block_norm_backward":
            s["workspace"] = torch.empty(max(1, binding.block_norm_backward_workspace_size(sh)),
                                         dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- the plain forms

def _sigmoid(z):
    return 1 / (1 + (-z).exp())


def _plain_linear(s):
    c = s["case"]
    N = c["N"]
    z = s["x"].float() @ s["w"].float()
    if s["bias"] is not None:
        z = z + s["bias"]
    if c["act"] == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif c["act"] == "gelu":
        z = z * _sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    elif c["act"] == "silu":
        z = z * _sigmoid(z)
    elif c["act"] == "swiglu":
        z = z[:, :N] * _sigmoid(z[:, :N]) * z[:, N:]
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z if c["fp32"] else z.to(torch.bfloat16)


def _plain_linear_backward(s):
    c = s["case"]
    N, d = c["N"], s["d_out"].float()
    z = s["preact"].float() if s["preact"] is not None else None
    if c["act"] == "relu":
        d = torch.where(z > 0, d, torch.zeros_like(d))
    elif c["act"] == "gelu":
        a = 2 * math.sqrt(2 / math.pi)
        p = _sigmoid(a * (z + 0.044715 * z * z * z))
        d = d * (p + z * p * (1 - p) * a * (1 + 3 * 0.044715 * z * z))
    elif c["act"] == "silu":
        p = _sigmoid(z)
        d = d * p * (1 + z * (1 - p))
    elif c["act"] == "swiglu":
        gate, up = z[:, :N], z[:, N:]
        p = _sigmoid(gate)
        d = torch.cat([d * up * p * (1 + gate * (1 - p)), d * gate * p], 1)
    out = {"d_x": (d @ s["w"].float().T).to(torch.bfloat16), "d_w": (s["x"].float().T @ d).to(torch.bfloat16)}
    if s["bias"] is not None:
        out["d_bias"] = d.sum(0)
    return out


def _gate(s):
    c = s["case"]
    return 1.0 if s["gate"] is None else s["gate"].float()[:, None] if c["gate"] == "token" else s["gate"].float()


def _plain_norm(s):
    c = s["case"]
    b = s["y"].float()
    if s["w_post"] is not None:
        b = b * ((b * b).mean(1, keepdim=True) + 1e-6).rsqrt() * (s["w_post"].float() + c["offset"])
    r = c["scale"] * s["x"].float() + _gate(s) * b
    out = {"residual": r.to(torch.bfloat16)}
    if s["w_pre"] is not None:
        z = r * ((r * r).mean(1, keepdim=True) + 1e-6).rsqrt() * (s["w_pre"].float() + c["offset"])
        out["normed"] = z.to(torch.bfloat16)
    return out


def _plain_norm_backward(s):
    c = s["case"]
    out, D, b = {}, s["d_r"].float(), s["y"].float()
    if s["w_pre"] is not None:
        r, dz = s["r"].float(), s["d_z"].float()
        rho = ((r * r).mean(1, keepdim=True) + 1e-6).rsqrt()
        hat, q = r * rho, dz * (s["w_pre"].float() + c["offset"])
        D = D + rho * (q - hat * (q * hat).mean(1, keepdim=True))
        out["d_pre"] = (dz * hat).sum(0)
    out["d_x"] = (c["scale"] * D).to(torch.bfloat16)
    d = _gate(s) * D
    if s["w_post"] is not None:
        w = s["w_post"].float() + c["offset"]
        sigma = ((b * b).mean(1, keepdim=True) + 1e-6).rsqrt()
        hat = b * sigma
        out["d_post"] = (d * hat).sum(0)
        b, h = hat * w, d * w
        d = sigma * (h - hat * (h * hat).mean(1, keepdim=True))
    out["d_y"] = d.to(torch.bfloat16)
    if s["gate"] is not None:
        out["d_gate"] = (D * b).sum(1 if c["gate"] == "token" else 0)
    return out


def _plain_clip(s):
    total = sum((x.float() * x.float()).sum().double() for x in s["grads"])
    norm = total.sqrt()
    by = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return {"norm": norm.float().view(1), "grads": [(x.float() * by).to(x.dtype) for x in s["grads"]]}


# ---------------------------------------------------------------- one pass

def _own_run(s):
    from mixture_experts_layer_up_amd import binding
    c = s["case"]
    if c["op"] == "linear":
        return binding.linear(s["shape"], s["x"], s["w"], bias=s["bias"], residual=s["residual"],
                              workspace=s["workspace"])
    if c["op"] == "linear_backward":
        d = binding.linear_backward(s["shape"], s["x"], s["w"], s["d_out"], preact=s["preact"],
                                    bias_grad=c["bias"], workspace=s["workspace"])
        return {k: v for k, v in d.items() if v is not None}
    if c["op"] == "clip_gradients":
        norm, grads = binding.clip_gradients(s["grads"], s["max_norm"], out=s["out"], workspace=s["workspace"])
        return {"norm": norm, "grads": grads}
    if c["op"] == "block_norm":
        r, z = binding.block_norm(s["shape"], s["x"], s["y"], post_weight=s["w_post"], pre_weight=s["w_pre"],
                                  gate=s["gate"])
        return {"residual": r} if z is None else {"residual": r, "normed": z}
    d = binding.block_norm_backward(s["shape"], s["r"], s["y"], post_weight=s["w_post"], pre_weight=s["w_pre"],
                                    gate=s["gate"], d_residual=s["d_r"], d_normed=s["d_z"],
                                    workspace=s["workspace"])
    names = {"d_x": "residual", "d_y": "branch", "d_post": "post_weight", "d_pre": "pre_weight", "d_gate": "gate"}
    return {k: d[v] for k, v in names.items() if d[v] is not None}


def run(state):
    if own:
        return _own_run(state)
    return {"linear": _plain_linear, "linear_backward": _plain_linear_backward, "block_norm": _plain_norm,
            "block_norm_backward": _plain_norm_backward, "clip_gradients": _plain_clip}[state["case"]["op"]](state)


def work(case):
    c = case
    if c["op"] in ("linear", "linear_backward"):
        M, K, N, W = c["M"], c["K"], c["N"], _width(c)
        out = M * N * (4 if c["fp32"] else 2)
        both = 2 * (M * K + K * W)
        if c["op"] == "linear":
            extra = (4 * W if c["bias"] else 0) + (2 * M * N if c["residual"] else 0)
            return {"bytes": both + out + extra, "flops": 2 * M * K * W}
        extra = (4 * W if c["bias"] else 0) + (2 * M * W if c["act"] != "none" else 0)
        return {"bytes": 2 * both + out + extra, "flops": 4 * M * K * W}
    if c["op"] == "clip_gradients":
        sizes, few = _sizes(c), _count_bf16(c)
        whole = c["tensors"] - few
        n = sum(sizes)
        return {"bytes": 8 * sum(sizes[:whole]) + 4 * sum(sizes[whole:]), "flops": 3 * n}
    T, H = c["T"], c["H"]
    gate = {"none": 0, "token": 4 * T, "channel": 2 * H}[c["gate"]]
    weights = 2 * H * (c["post"] + c["pre"])
    if c["op"] == "block_norm":
        return {"bytes": 2 * T * H * (3 + c["pre"]) + gate + weights, "flops": T * H * 10}
    # the branch is read only where a weight, a gate or its norm needs it
    arrays = 3 + 2 * c["pre"] + (1 if c["post"] or c["gate"] != "none" else 0)
    grads = 4 * H * (c["post"] + c["pre"] + (c["gate"] == "channel")) + (4 * T if c["gate"] == "token" else 0)
    return {"bytes": 2 * T * H * arrays + gate + weights + grads, "flops": T * H * 25}


# ---------------------------------------------------------------- the definition in 64 bits

def _act(name, z, N):
    """The activation of float64 pre-activations, by its definition."""
    if name == "relu":
        return torch.clamp(z, min=0.0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "swiglu":
        return z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:]
    return z


def _rms(x):
    return x / torch.sqrt((x ** 2).sum(1, keepdim=True) / x.shape[1] + 1e-6)


def _block(c, x, y, w_post, w_pre, gate):
    """(new residual, normed or None) in float64, differentiable."""
    b = y if w_post is None else _rms(y) * (w_post + c["offset"])
    if gate is not None:
        b = b * (gate[:, None] if c["gate"] == "token" else gate)
    r = x * c["scale"] + b
    return r, None if w_pre is None else _rms(r) * (w_pre + c["offset"])


def _leaf(t):
    return None if t is None else t.double().requires_grad_()


def _exact_norm_backward(s, c):
    """By automatic differentiation: the second norm at the stored residual stream, the first part below it."""
    out = {}
    D = s["d_r"].double()
    if s["w_pre"] is not None:
        r, w = _leaf(s["r"]), _leaf(s["w_pre"])
        d_r, out["d_pre"] = torch.autograd.grad(_rms(r) * (w + c["offset"]), (r, w), s["d_z"].double())
        D = D + d_r
    x, y, w, gate = _leaf(s["x"]), _leaf(s["y"]), _leaf(s["w_post"]), _leaf(s["gate"])
    at = [t for t in (x, y, w, gate) if t is not None]
    got = iter(torch.autograd.grad(_block(c, x, y, w, None, gate)[0], at, D))
    out["d_x"] = next(got)
    d_y = next(got)
    if w is not None:
        out["d_post"] = next(got)
    out["d_y"] = d_y
    if gate is not None:
        out["d_gate"] = next(got)
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "clip_gradients":
        flat = torch.cat([x.double().view(-1) for x in s["grads"]])
        norm = torch.linalg.vector_norm(flat)
        by = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
        return {"norm": norm.view(1), "grads": [x.double() * by for x in s["grads"]]}
    if c["op"] == "block_norm":
        wide = {k: None if s[k] is None else s[k].double() for k in ("x", "y", "w_post", "w_pre", "gate")}
        r, z = _block(c, **wide)
        return {"residual": r} if z is None else {"residual": r, "normed": z}
    if c["op"] == "block_norm_backward":
        return _exact_norm_backward(s, c)
    x, w = s["x"].double(), s["w"].double()
    if c["op"] == "linear":
        z = x @ w if s["bias"] is None else torch.addmm(s["bias"].double(), x, w)
        z = _act(c["act"], z, c["N"])
        return z if s["residual"] is None else z + s["residual"].double()
    d = s["d_out"].double()
    if c["act"] != "none":
        z = s["preact"].double().requires_grad_()
        d, = torch.autograd.grad(_act(c["act"], z, c["N"]), z, d)
    out = {"d_x": torch.mm(d, w.T), "d_w": torch.mm(x.T, d)}
    if c["bias"]:
        out["d_bias"] = d.sum(0)
    return out
