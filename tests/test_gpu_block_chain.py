"""The products, norms and clipping together with the layer, as a block in training
runs them; captured, replayed, and on streams of their own."""
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _block
from tests._gpu import announce

pytestmark = pytest.mark.gpu

T, H, I, E, K, EPS = 200, 256, 96, 16, 4, 1e-6


class Block:
    """One block: norm, router, 4-bit routed experts and a shared expert, norm."""

    def __init__(self, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.x, self.y = r(T, H).bfloat16(), r(T, H).bfloat16()
        self.w_in, self.w_out = (1 + 0.2 * r(H)).bfloat16(), (1 + 0.2 * r(H)).bfloat16()
        self.w_next, self.gate = (1 + 0.2 * r(H)).bfloat16(), (0.5 * r(H)).bfloat16()
        self.router, self.router_bias = (0.1 * r(H, E)).bfloat16(), 0.1 * r(E)
        self.s13, self.s2 = (0.06 * r(H, 2 * I)).bfloat16(), (0.1 * r(I, H)).bfloat16()
        self.d_r, self.d_z = (0.1 * r(T, H)).bfloat16(), (0.1 * r(T, H)).bfloat16()
        self.shape = binding.Shape(T, H, I, E, K, 0, E, 0, 0, 0, 1.0, 0, 0)
        self.fmt = binding.W4Format(32, 0)
        w13, w2 = (0.06 * r(E, H, 2 * I)).bfloat16(), (0.1 * r(E, I, H)).bfloat16()
        self.experts = binding.pack_weights_w4(self.shape, self.fmt,
                                               *binding.quantize_w4(self.shape, self.fmt, w13, w2))
        self.norm = binding.NormShape(T, H, EPS, 1.0, 0.0, 0)
        self.gated = binding.NormShape(T, H, EPS, 0.5, 0.0, 2)
        self.logits_of = binding.LinearShape(T, H, E, 0, 1)
        self.up = binding.LinearShape(T, H, I, 4, 0)
        self.down = binding.LinearShape(T, I, H, 0, 0)

    def forward(self):
        s = {}
        s["r0"], s["h"] = binding.block_norm(self.norm, self.x, self.y, pre_weight=self.w_in)
        s["logits"] = binding.linear(self.logits_of, s["h"], self.router, bias=self.router_bias)
        s["routing"] = binding.alloc_routing(self.shape, "cuda")
        s["rows"] = torch.zeros((T * K, H), dtype=torch.bfloat16, device="cuda")
        binding.forward_w4(self.shape, self.fmt, s["h"], *self.experts, router_logits=s["logits"],
                           routing=s["routing"], expert_out=s["rows"])
        s["routed"] = binding.finalize(self.shape, s["rows"], s["routing"])
        s["pre"] = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
        s["act"] = binding.linear(self.up, s["h"], self.s13, preact=s["pre"])
        # the shared expert's output on top of the routed one, in place
        s["out"] = binding.linear(self.down, s["act"], self.s2, residual=s["routed"], out=s["routed"].clone())
        s["r1"], s["z"] = binding.block_norm(self.gated, s["r0"], s["out"], post_weight=self.w_out,
                                             pre_weight=self.w_next, gate=self.gate)
        return s

    def backward(self, s):
        d = {}
        d["norm"] = binding.block_norm_backward(self.gated, s["r1"], s["out"], post_weight=self.w_out,
                                                pre_weight=self.w_next, gate=self.gate, d_residual=self.d_r,
                                                d_normed=self.d_z)
        d_out = d["norm"]["branch"]
        d["down"] = binding.linear_backward(self.down, s["act"], self.s2, d_out)
        d["up"] = binding.linear_backward(self.up, s["h"], self.s13, d["down"]["d_x"], preact=s["pre"])
        d["rows"], d["weights"] = binding.finalize_backward(self.shape, d_out, s["rows"], s["routing"])
        bal = binding.balance_loss(self.shape, s["logits"], s["routing"]["topk_ids"])
        d["logits"] = binding.route_backward(self.shape, s["logits"], s["routing"]["topk_ids"],
                                             s["routing"]["topk_weights"], d["weights"], balance=bal,
                                             d_loss=torch.full((1,), 0.01, device="cuda"))
        d["router"] = binding.linear_backward(self.logits_of, s["h"], self.router, d["logits"], bias_grad=True)
        d_h = (d["up"]["d_x"].float() + d["router"]["d_x"].float()).bfloat16()
        d["d_h"] = d_h
        d["first"] = binding.block_norm_backward(self.norm, s["r0"], self.y, pre_weight=self.w_in,
                                                 d_residual=d["norm"]["residual"], d_normed=d_h)
        d["grads"] = [d["norm"]["post_weight"], d["norm"]["pre_weight"], d["norm"]["gate"], d["first"]["pre_weight"],
                      d["up"]["d_w"], d["down"]["d_w"], d["router"]["d_w"], d["router"]["d_bias"]]
        d["clipped_norm"], d["clipped"] = binding.clip_gradients(d["grads"], 0.1,
                                                                 out=[torch.empty_like(g) for g in d["grads"]])
        return d


def test_block_in_training():
    """Every step against float64 on the inputs that the step before made."""
    announce("block in training")
    b = Block(1)
    s = b.forward()
    d = b.backward(s)

    def near(got, want, bound):
        assert _block.worst(got, want, bound) <= 1

    r, off, z, off_z = _block.norm(b.x, b.y, None, b.w_in, None, EPS, 1.0, 0.0)
    near(s["r0"], r, off)
    near(s["h"], z, off_z)
    near(s["logits"], *_block.linear(s["h"], b.router, "none", b.router_bias, None, True)[:2])
    out, off, pre, off_pre = _block.linear(s["h"], b.s13, "swiglu")
    near(s["act"], out, off)
    near(s["pre"], pre, off_pre)
    near(s["out"], *_block.linear(s["act"], b.s2, "none", None, s["routed"])[:2])
    r, off, z, off_z = _block.norm(s["r0"], s["out"], b.w_out, b.w_next, b.gate, EPS, 0.5, 0.0)
    near(s["r1"], r, off)
    near(s["z"], z, off_z)
    want = _block.norm_backward(s["r1"], s["out"], b.w_out, b.w_next, b.gate, b.d_r, b.d_z, EPS, 0.5, 0.0, False)
    for k, v in d["norm"].items():
        near(v, *want[k])
    for name, w, x, d_out, act, pre in (("down", b.s2, s["act"], d["norm"]["branch"], "none", None),
                                        ("up", b.s13, s["h"], d["down"]["d_x"], "swiglu", s["pre"]),
                                        ("router", b.router, s["h"], d["logits"], "none", None)):
        want = _block.linear_backward(x, w, d_out, act, pre)
        for k, v in d[name].items():
            if v is not None:
                near(v, *want[k])
    want = _block.norm_backward(s["r0"], b.y, None, b.w_in, None, d["norm"]["residual"], d["d_h"], EPS, 1.0, 0.0, False)
    for k in ("residual", "branch", "pre_weight"):
        near(d["first"][k], *want[k])
    total, f, scaled = _block.clip(d["grads"], 0.1)
    assert f < 1 and abs(float(d["clipped_norm"]) - total) <= 2 * _block.U32 * total
    for got, w in zip(d["clipped"], scaled):
        near(got, w, ((_block.U16 if got.dtype == torch.bfloat16 else _block.U32) + 4 * _block.U32) * w.abs() + 1e-30)


def _flat(tree):
    if isinstance(tree, torch.Tensor):
        return [tree]
    if isinstance(tree, dict):
        tree = list(tree.values())
    return [t for v in tree or () for t in _flat(v)] if isinstance(tree, (list, tuple)) else []


def test_captured_and_replayed():
    """Forward, backward and clipping in one graph, replayed on other inputs with eager work
    and other memory between the replays: each replay is bitwise the eager pass."""
    announce("block captured")
    b = Block(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.backward(b.forward())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = b.forward()
        d = b.backward(s)
    for turn in range(4):
        g = torch.Generator("cuda").manual_seed(50 + turn)
        b.x.copy_(torch.randn((T, H), generator=g, device="cuda"))
        b.d_z.copy_(torch.randn((T, H), generator=g, device="cuda") * 0.1)
        graph.replay()
        junk = torch.randn(1 << 20, device="cuda", generator=g).sum().item()
        torch.cuda.synchronize()
        eager_s = b.forward()
        eager_d = b.backward(eager_s)
        assert junk == junk
        for name in ("r0", "h", "logits", "routed", "act", "pre", "out", "r1", "z"):
            assert torch.equal(s[name], eager_s[name]), (turn, name)
        for name in d:
            for one, two in zip(_flat(d[name]), _flat(eager_d[name])):
                assert torch.equal(one, two), (turn, name)


def test_two_graphs_on_two_streams():
    """Two captured passes with workspaces of their own run at once."""
    announce("two captured products")
    M, K_, N = 700, 1024, 136
    g = torch.Generator("cuda").manual_seed(3)
    sh = binding.LinearShape(M, K_, N, 0, 0)
    runs = []
    for _ in range(2):
        x = torch.randn((M, K_), generator=g, device="cuda").bfloat16()
        w = torch.randn((K_, N), generator=g, device="cuda").bfloat16()
        ws = torch.empty(max(1, binding.linear_workspace_size(sh)), dtype=torch.uint8, device="cuda")
        want = binding.linear(sh, x, w)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(5):
                binding.linear(sh, x, w, out=out, workspace=ws)
        runs.append((graph, stream, out, want, (x, w, ws)))     # the graph reads them
    for _ in range(3):
        for graph, stream, out, *_ in runs:
            with torch.cuda.stream(stream):
                out.zero_()
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, _, out, want, _ in runs)


def test_current_stream_is_used():
    """Work on another stream follows that stream's order."""
    announce("block on another stream")
    b = Block(4)
    want = b.forward()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        keep, b.x = b.x, torch.zeros_like(b.x)
        a = torch.randn((4096, 4096), device="cuda")
        for _ in range(20):
            a = a @ a * 1e-3     # keeps the stream busy
        b.x.copy_(keep)
        got = b.forward()
    stream.synchronize()
    for name in ("r0", "logits", "out", "r1", "z"):
        assert torch.equal(got[name], want[name])


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, shape):
        ctx.shape = shape
        pre = torch.empty((shape.rows, 2 * shape.out_features), dtype=torch.bfloat16, device=x.device)
        out = binding.linear(shape, x, w, preact=pre)
        ctx.save_for_backward(x, w, pre)
        return out

    @staticmethod
    def backward(ctx, d):
        x, w, pre = ctx.saved_tensors
        got = binding.linear_backward(ctx.shape, x, w, d.contiguous(), preact=pre)
        return got["d_x"], got["d_w"], None


def test_autograd_function_around_a_product():
    """As a torch user wraps it: a broadcast gradient arrives and is made contiguous."""
    announce("linear in autograd")
    g = torch.Generator("cuda").manual_seed(6)
    sh = binding.LinearShape(50, 64, 24, 4, 0)
    x = torch.randn((50, 64), generator=g, device="cuda").bfloat16().requires_grad_()
    w = (torch.randn((64, 48), generator=g, device="cuda") * 0.2).bfloat16().requires_grad_()
    out = _Linear.apply(x, w, sh)
    out.sum().backward()
    pre = _block.linear(x.detach(), w.detach(), "none")[2].bfloat16()
    want = _block.linear_backward(x.detach(), w.detach(), torch.ones((50, 24), device="cuda").bfloat16(), "swiglu", pre)
    # pre is rounded from float64 here: where fp32 rounds it to a neighbour, dz moves by a step of it
    step = {k: 2 * off for k, (_, off) in want.items()}
    assert _block.worst(x.grad, want["d_x"][0], step["d_x"]) <= 1
    assert _block.worst(w.grad, want["d_w"][0], step["d_w"]) <= 1


def test_bindings_refuse():
    sh = binding.LinearShape(8, 64, 24, 0, 0)
    x = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((64, 24), dtype=torch.bfloat16, device="cuda")
    for kw, what in ((dict(x=x.float()), "dtype"), (dict(x=x[:4]), "shape"), (dict(w=w.T), "contiguous"),
                     (dict(w=w.cpu()), "one GPU"), (dict(bias=torch.zeros(24, dtype=torch.bfloat16, device="cuda")), "dtype"),
                     (dict(residual=torch.zeros((8, 25), dtype=torch.bfloat16, device="cuda")), "shape"),
                     (dict(out=torch.zeros((8, 24), device="cuda")), "dtype")):
        args = dict(x=x, w=w)
        args.update(kw)
        with pytest.raises(binding.MoELoRAError, match=what):
            binding.linear(sh, **args)
    d = torch.zeros((8, 24), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.MoELoRAError, match="invalid"):
        binding.linear_backward(sh, None, w, d)
    with pytest.raises(binding.MoELoRAError, match="invalid"):
        binding.linear_backward(sh, x, w, d, x_grad=False, w_grad=False)
    with pytest.raises(binding.MoELoRAError, match="workspace"):
        big = binding.LinearShape(8, 64, 25, 0, 0)
        binding.linear_backward(big, x, torch.zeros((64, 25), dtype=torch.bfloat16, device="cuda"),
                                torch.zeros((8, 25), dtype=torch.bfloat16, device="cuda"),
                                workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    nm = binding.NormShape(8, 64, 1e-6, 1.0, 0.0, 0)
    v = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    for args, kw, what in (((None, None), {}, "must be given"), ((x, None), dict(post_weight=v), "invalid"),
                           ((x, x), dict(pre_weight=v.float()), "dtype"), ((x, x[:3]), {}, "shape"),
                           ((x, x), dict(gate=v), "invalid")):
        with pytest.raises(binding.MoELoRAError, match=what):
            binding.block_norm(nm, *args, **kw)
    with pytest.raises(binding.MoELoRAError, match="must be given"):
        binding.block_norm_backward(nm, x, x)
