"""The layer with 4-bit expert weights on the GPU against its definition in
float64, every output row, within the bound of its stated roundings."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _w4
from tests._gpu import SideStream, announce, bf16_to_np, tol
from tests._w4 import W4Case

pytestmark = pytest.mark.gpu

CASES = [
    W4Case("one_token", 1, 128, 64, 8, 2, L=1, rg=8, rd=8),
    W4Case("one_expert_one_row", 1, 64, 32, 1, 1, group=32),
    W4Case("smallest_sizes_zeros", 5, 64, 32, 3, 2, group=64, zeros=1),
    W4Case("group_past_k", 9, 64, 96, 4, 2, group=128, zeros=1),
    W4Case("k_not_unit_multiple", 20, 192, 96, 6, 3, L=2, rg=4, rd=12, group=32, zeros=1),
    W4Case("last_group_short", 20, 320, 160, 6, 3, L=3, rg=16, rd=16, group=128),
    W4Case("group64_short", 33, 192, 224, 5, 2, L=1, rg=20, rd=4, group=64, zeros=1),
    W4Case("shard", 40, 256, 128, 16, 4, off=5, E_l=6, L=2, rg=8, rd=8, scaling=2.5),
    W4Case("shard_without_slots", 3, 128, 64, 64, 2, off=63, E_l=1, seed=4),
    W4Case("method1_odd_rank", 24, 128, 64, 8, 3, L=3, rg=5, rd=7, method=1),
    W4Case("shared_outer", 30, 256, 96, 8, 2, L=2, rg=16, rd=8, shared=1, group=32),
    W4Case("rank_zero_down", 12, 128, 64, 4, 2, L=2, rg=8, rd=0),
    W4Case("rows16_to_48", 60, 256, 128, 4, 2, L=2, rg=16, rd=16),
    W4Case("two_tiles_an_expert", 130, 192, 96, 3, 2, L=1, rg=8, rd=24, zeros=1, group=32),
    W4Case("many_rows", 150, 256, 128, 2, 1, L=2, rg=64, rd=64),
    W4Case("many_rows_odd", 211, 192, 160, 3, 2, L=2, rg=8, rd=16, zeros=1, group=64),
    W4Case("more_than_one_slot_block", 300, 128, 64, 16, 4, L=2, rg=8, rd=8),
]


def _run(c, x, **over):
    shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
    kw["router_logits"] = logits
    kw.update(over)
    out = binding.forward_w4(shape, fmt, hidden, *packed, **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
def test_forward_w4_matches_definition(c):
    announce(f"forward_w4 {c}")
    x = _w4.inputs(c)
    got = bf16_to_np(_run(c, x))
    ref, bound, _ = _w4.reference(c, x)
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), f"{(over > 0).sum()} of {over.size} outside, worst {over.max():.3e}"
    assert np.abs(got - ref).max(initial=0.0) <= tol(ref)


def _draw(i):
    rng = np.random.default_rng(300 + i)
    E = int(rng.integers(1, 24))
    k = int(rng.integers(1, min(6, E) + 1))
    E_l = int(rng.integers(1, E + 1))
    rank = lambda: int(rng.choice([0, 1, 4, 8, 12, 16, 40, 64]))  # noqa: E731
    return W4Case(f"rand{i}", int(np.exp(rng.uniform(0, np.log(250)))), 64 * int(rng.integers(1, 6)),
                  32 * int(rng.integers(1, 8)), E, k, int(rng.integers(0, E - E_l + 1)), E_l,
                  int(rng.integers(0, 4)), rank(), rank(), int(rng.choice([32, 64, 128])),
                  int(rng.integers(0, 2)), int(rng.integers(0, 2)), float(rng.choice([1.0, 0.5])),
                  int(rng.random() < 0.25), 700 + i)


# Tiles of 64 rows (many slots) with experts that fill one to four row tiles,
# K of several staged panels and an odd number of steps, the largest ranks and
# adapter counts.
LARGE = [
    W4Case("tiles64", 4100, 128, 64, 3, 1, L=2, rg=16, rd=40),
    W4Case("tiles64_few_rows_each", 1400, 320, 32, 100, 3, L=2, rg=8, rd=8, group=64),
    W4Case("tiles64_zeros32", 2060, 192, 96, 24, 2, L=1, rg=8, rd=8, zeros=1, group=32),
    W4Case("tiles64_rank256", 4100, 64, 64, 2, 1, L=2, rg=256, rd=256, zeros=1, group=64),
    W4Case("tiles64_shared_odd_ranks", 2100, 128, 64, 8, 2, L=3, rg=13, rd=22, shared=1, group=32),
    W4Case("tiles64_no_lora", 4200, 64, 32, 4, 1, zeros=1),
    W4Case("tiles32_long_k", 400, 1216, 1088, 2, 1, L=1, rg=72, rd=8, group=64),
    W4Case("tiles32_rank256", 300, 128, 64, 4, 2, L=2, rg=256, rd=200),
    W4Case("panels_8_waves", 1, 4224, 1056, 4, 2, L=1, rg=40, rd=256, zeros=1, group=32),
    W4Case("panels_4_waves", 60, 2240, 1120, 16, 2, L=2, rg=256, rd=36, group=64),
    W4Case("adapters64", 200, 128, 64, 4, 2, L=64, rg=8, rd=8),
    W4Case("adapters64_few_rows", 40, 128, 64, 8, 2, L=64, rg=36, rd=8, zeros=1, group=32),
]


@pytest.mark.parametrize("c", LARGE, ids=lambda c: c.name)
def test_forward_w4_large(c):
    test_forward_w4_matches_definition(c)


@pytest.mark.parametrize("c", [_draw(i) for i in range(16)], ids=lambda c: c.name)
def test_forward_w4_random_shapes(c):
    test_forward_w4_matches_definition(c)


def test_forward_w4_given_topk_and_flags():
    """Given ids: out-of-range ones are slots of no expert, the same expert twice
    counts twice, and the flag word names bad values."""
    c = W4Case("given", 17, 128, 64, 6, 3, L=2, rg=8, rd=8, seed=9)
    x = _w4.inputs(c)
    ids, w = _w4.route(c, x["logits"])
    ids = ids.astype(np.int32)
    ids[2], ids[3, 1], ids[4], ids[5, 2] = -1, 77, [1, 1, 1], -9
    x["mapping"][6] = 5
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    announce("forward_w4 given top-k")
    got = bf16_to_np(_run(c, x, router_logits=None, topk_ids=torch.from_numpy(ids).cuda(),
                          topk_weights=torch.from_numpy(w.astype(np.float32)).cuda(),
                          input_flags=flags))
    ref, bound, _ = _w4.reference(c, x, ids, w.astype(np.float32).astype(np.float64))
    assert (np.abs(got - ref) <= bound).all()
    assert (got[2] == 0).all()
    assert int(flags) == binding.FLAG_EXPERT_ID | binding.FLAG_ADAPTER


@pytest.mark.parametrize("T", [5, 150])
def test_forward_w4_expert_out_and_finalize(T):
    """expert_out holds the slots' outputs at their rows, rows past the local slots
    stay as they were, and finalize of them is out within their rounding."""
    c = W4Case("expert_out", T, 192, 96, 6, 2, off=1, E_l=3, L=1, rg=8, rd=8, zeros=1, group=64)
    x = _w4.inputs(c)
    shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
    announce(f"forward_w4 expert_out T={T}")
    rows = torch.full((c.T * c.k, c.H), 7.0, dtype=torch.bfloat16, device="cuda")
    r = binding.alloc_routing(shape, "cuda")
    assert binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, routing=r,
                              expert_out=rows, **kw) is None
    out = binding.finalize(shape, rows, r)
    whole = binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, **kw)
    torch.cuda.synchronize()
    ref, bound, slots = _w4.reference(c, x)
    ids, w = _w4.route(c, x["logits"])
    perm = r["expanded_idx_to_permuted_idx"].cpu().numpy()
    got = bf16_to_np(rows)
    P = int(r["expert_offsets"][-1])
    assert (got[P:] == 7.0).all()
    extra = np.zeros_like(bound)
    for (t, j), y in slots.items():
        extra[t] += w[t, j] * _w4.U * (np.abs(y) + bound[t])
    assert (np.abs(bf16_to_np(out) - ref) <= bound + extra).all()
    assert (np.abs(bf16_to_np(whole) - ref) <= bound).all()
    for (t, j), y in slots.items():
        p = perm[t * c.k + j]
        assert 0 <= p < P
        # one slot's own bound: that of a layer with this slot alone
        one = np.full((c.T, c.k), -1)
        one[t, j] = ids[t, j]
        if t < 3:
            _, b1, _ = _w4.reference(c, x, one, np.ones((c.T, c.k)))
            assert (np.abs(got[p] - y) <= b1[t]).all()


def test_forward_w4_empty_batch_and_no_local_slot():
    c = W4Case("empty", 0, 128, 64, 4, 2)
    x = _w4.inputs(c)
    announce("forward_w4 empty batch")
    assert _run(c, x).shape == (0, 128)


def test_forward_w4_graph_replays_and_streams():
    """Captured on a side stream and replayed with eager work between, two
    captured forwards with workspaces of their own; every replay is the eager
    result bit for bit, as is the two-stream schedule."""
    c = W4Case("graph", 40, 256, 128, 16, 4, L=2, rg=16, rd=8, zeros=1, group=64)
    x = _w4.inputs(c)
    shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
    announce("forward_w4 graph")
    eager = binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, **kw)
    size = binding.workspace_size_w4(shape, fmt)
    outs, graphs, spaces = [], [], []
    for _ in range(2):
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(eager)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, out=out,
                               workspace=ws, **kw)
        outs.append(out), graphs.append(g), spaces.append(ws)
    for _ in range(3):
        for out, ws in zip(outs, spaces):
            out.fill_(float("nan"))
            ws.fill_(0xff)
        graphs[0].replay()
        graphs[1].replay()
        between = binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, **kw)
        torch.cuda.synchronize()
        for o in (*outs, between):
            assert torch.equal(o, eager)
    side = SideStream()
    two = binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, **side.kwargs(), **kw)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        elsewhere = binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, **kw)
    torch.cuda.synchronize()
    side.close()
    assert torch.equal(two, eager) and torch.equal(elsewhere, eager)


@pytest.mark.parametrize("zeros", [0, 1])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_w4(zeros, group):
    """Scales, zero points and codes as defined, and weights within half a step
    plus what rounding the step to bf16 moves the ends."""
    shape = binding.Shape(1, 192, 96, 3, 1, 0, 3, 0, 0, 0, 1.0, 0, 0)
    fmt = binding.W4Format(group, zeros)
    g = torch.Generator().manual_seed(5)
    ws = [(torch.randn(s, generator=g) * 0.02).to(torch.bfloat16) for s in ((3, 192, 192), (3, 96, 192))]
    ws[0][0, :, 3] = 0.0                       # groups of zeros
    ws[0][1, :, 4] = ws[0][1, :, 4].abs()      # one-sided groups
    ws[0][1, :, 5] = -ws[0][1, :, 5].abs()
    announce(f"quantize_w4 {group} {zeros}")
    for w, q in zip(ws, binding.quantize_w4(shape, fmt, *(w.cuda() for w in ws))):
        E, K, N = w.shape
        codes, s = q["codes"].cpu().numpy(), q["scales"].float().cpu().numpy()
        z = q["zeros"].cpu().numpy().astype(np.float32) if zeros else np.full(s.shape, 8, np.float32)
        wn = w.float().numpy()
        for b in range(s.shape[1]):
            part = wn[:, b * group:(b + 1) * group]
            lo, hi = np.minimum(part.min(1), 0), np.maximum(part.max(1), 0)
            step = (hi.astype(np.float64) - lo) / 15 if zeros else np.maximum(hi, -lo) / 7.0
            assert (np.abs(s[:, b] - step) <= _w4.U * step * (1 + 2.0 ** -20)).all()
            with np.errstate(invalid="ignore", divide="ignore"):
                if zeros:
                    want = np.clip(np.rint(-lo / s[:, b]), 0, 15)
                    assert (np.where(s[:, b] > 0, z[:, b] == want, z[:, b] == 0)).all()
                q_want = np.clip(np.rint(part / s[:, b][:, None]) + z[:, b][:, None], 0, 15)
            q_want = np.where(s[:, b][:, None] > 0, q_want, z[:, b][:, None])
            k0 = b * group
            got = np.empty_like(part)
            rows = codes[:, k0 // 2:(k0 + part.shape[1]) // 2]
            got[:, 0::2], got[:, 1::2] = rows & 15, rows >> 4
            assert (got == q_want).all()
        back = _w4.dequantise({"codes": codes, "scales": s, "zeros": z.astype(np.uint8)}, group)
        big = s[:, np.arange(K) // group]
        # half a step, the ends' shortfall of 7 U or 15 U steps, a rounded zero point's half step
        assert (np.abs(back - wn) <= big * ((1.0 if zeros else 0.5) + 15 * _w4.U)).all()


def test_forward_w4_of_quantised_weights_is_near_bf16_forward():
    """quantize_w4 -> pack -> forward_w4 against the layer of the dequantised
    weights: the whole load path."""
    c = W4Case("quantised", 30, 256, 128, 8, 2, L=1, rg=8, rd=8, zeros=1, group=64)
    x = _w4.inputs(c)
    g = torch.Generator().manual_seed(3)
    w13 = (torch.randn((8, 256, 256), generator=g) * 0.05).to(torch.bfloat16)
    w2 = (torch.randn((8, 128, 256), generator=g) * 0.05).to(torch.bfloat16)
    announce("quantize_w4 -> forward_w4")
    shape, fmt, hidden, _, kw, logits = _w4.device_layer(c, x)
    q = binding.quantize_w4(shape, fmt, w13.cuda(), w2.cuda())
    packed = binding.pack_weights_w4(shape, fmt, *q)
    got = bf16_to_np(binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, **kw))
    for name, d in zip(("w13", "w2"), q):
        x[name] = {"codes": d["codes"].cpu().numpy(), "scales": d["scales"].float().cpu().numpy(),
                   "zeros": d["zeros"].cpu().numpy()}
    ref, bound, _ = _w4.reference(c, x)
    assert (np.abs(got - ref) <= bound).all()


def test_forward_w4_refusals_of_the_binding():
    c = W4Case("refuse", 4, 128, 64, 4, 2, zeros=1, group=64)
    x = _w4.inputs(c)
    shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
    call = lambda *a, **o: binding.forward_w4(shape, fmt, *a, **{**kw, "router_logits": logits, **o})  # noqa: E731
    with pytest.raises(binding.MoELoRAError, match="w13_packed"):
        call(hidden, packed[0][:-1], packed[1])
    with pytest.raises(binding.MoELoRAError, match="dtype"):
        call(hidden, packed[0].view(torch.int8), packed[1])
    with pytest.raises(binding.MoELoRAError, match="one GPU"):
        call(hidden, packed[0].cpu(), packed[1])
    with pytest.raises(binding.MoELoRAError, match="contiguous"):
        call(hidden.t().contiguous().t(), *packed)
    with pytest.raises(binding.MoELoRAError, match="workspace"):
        call(hidden, *packed, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    q = {"codes": torch.zeros((4, 64, 128), dtype=torch.uint8, device="cuda"),
         "scales": torch.zeros((4, 2, 128), dtype=torch.bfloat16, device="cuda")}
    with pytest.raises(binding.MoELoRAError, match="zeros"):
        binding.pack_weights_w4(shape, fmt, q, q)
