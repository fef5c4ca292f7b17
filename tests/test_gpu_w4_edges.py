"""The 4-bit layer without local slots and with an empty batch, and the training
entry points with device values out of range, which must only count as nothing."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _w4
from tests._gpu import announce
from tests._w4 import W4Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40, 700, 6000])
def test_shard_without_a_slot(T):
    """Every id belongs to another shard: zeros, whatever the hidden rows hold, and
    expert_out stays as it was."""
    c = W4Case("none", T, 128, 64, 16, 2, off=12, E_l=4, L=2, rg=8, rd=8, zeros=1, group=64)
    x = _w4.inputs(c)
    x["hidden"][:] = np.nan
    shape, fmt, hidden, packed, kw, _ = _w4.device_layer(c, x)
    kw["topk_ids"] = torch.randint(0, 12, (T, 2), dtype=torch.int32, device="cuda")
    kw["topk_weights"] = torch.full((T, 2), 0.5, device="cuda")
    announce(f"no local slot T={T}")
    out = torch.full((T, c.H), float("nan"), dtype=torch.bfloat16, device="cuda")
    binding.forward_w4(shape, fmt, hidden, *packed, out=out, **kw)
    assert (out == 0).all()
    rows = torch.full((T * 2, c.H), 3.0, dtype=torch.bfloat16, device="cuda")
    r = binding.alloc_routing(shape, "cuda")
    binding.forward_w4(shape, fmt, hidden, *packed, expert_out=rows, routing=r, **kw)
    assert (rows == 3.0).all() and int(r["expert_offsets"][-1]) == 0
    assert (r["expanded_idx_to_permuted_idx"] == -1).all()


def test_empty_batch():
    c = W4Case("empty", 0, 128, 64, 4, 2, L=1, rg=8, rd=8)
    x = _w4.inputs(c)
    shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
    announce("empty batch")
    r = binding.alloc_routing(shape, "cuda")
    for t in r.values():
        t.fill_(7)
    out = binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, routing=r, **kw)
    assert out.shape == (0, 128)
    for name in ("expert_counts", "expert_offsets", "lora_seg_offsets"):
        assert (r[name] == 0).all()
    bal = binding.balance_loss(shape, logits, torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                               seq_offsets=torch.zeros(21, dtype=torch.int32, device="cuda"))
    assert float(bal["loss"]) == 0 and bal["counts"].shape == (20, 4)
    assert all((bal[n] == 0).all() for n in ("counts", "probs", "tokens"))
    one = torch.ones(1, device="cuda")
    assert binding.route_backward(shape, logits, balance=bal, d_loss=one,
                                  seq_offsets=torch.zeros(21, dtype=torch.int32, device="cuda")).shape == (0, 4)


@pytest.mark.parametrize("T,E", [(40, 16), (3000, 96)])
def test_offsets_out_of_range_stay_inside_the_arrays(T, E):
    """Negative, descending and too large offsets: unspecified values, but nothing
    outside the outputs is written and tokens of no sequence have no gradient."""
    k, S, guard = 2, 9, 4096
    sh = binding.Shape(T, 64, 32, E, k, 0, E, 0, 0, 0, 1.0, 0, 0)
    x = torch.randn((T, E), device="cuda", generator=torch.Generator("cuda").manual_seed(0))
    ids = x.topk(k).indices.int()
    lib, ref = binding.load_library(), binding.ctypes.byref
    for off in ([5, -3, 2 ** 31 - 1, 0, T, -2 ** 31, 7, T + 9, 1, 0], [T] * 10, [-1] * 10,
                list(range(9, -1, -1)), [T, 0] * 5):
        offsets = torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda()
        sizes = {"loss": 1, "counts": S * E, "probs": S * E, "tokens": S, "d": T * E,
                 "ws": int(lib.moe_lora_balance_workspace_size(ref(sh), S)) // 4}
        buf = {n: torch.full((v + 2 * guard,), 0x7abcdef, dtype=torch.int32, device="cuda")
               for n, v in sizes.items()}
        p = {n: b.data_ptr() + 4 * guard for n, b in buf.items()}
        tokens = binding.Tokens(None, offsets.data_ptr(), S)
        bal = binding.Balance(p["loss"], p["counts"], p["probs"], p["tokens"])
        one = torch.ones(1, device="cuda")
        announce(f"offsets {off} T={T}")
        stream = torch.cuda.current_stream().cuda_stream
        assert lib.moe_lora_balance_loss(ref(sh), x.data_ptr(), ids.data_ptr(), ref(tokens), ref(bal), p["ws"],
                                         4 * sizes["ws"], stream) == 0
        assert lib.moe_lora_route_backward(ref(sh), x.data_ptr(), None, None, None, ref(tokens), ref(bal),
                                           one.data_ptr(), p["d"], stream) == 0
        torch.cuda.synchronize()
        for n, b in buf.items():
            assert (b[:guard] == 0x7abcdef).all() and (b[guard + sizes[n]:] == 0x7abcdef).all(), n
        if max(off) <= 0 or min(off) >= T:
            d = buf["d"][guard:guard + T * E]
            assert (d == 0).all() and float(buf["loss"][guard:guard + 1].view(torch.float32)) == 0


def test_permuted_indices_out_of_range_count_as_not_local():
    T, k, H = 30, 4, 192
    sh = binding.Shape(T, H, 32, 8, k, 0, 8, 0, 0, 0, 1.5, 0, 0)
    g = torch.Generator("cuda").manual_seed(1)
    d, y = (torch.randn((n, H), device="cuda", generator=g).bfloat16() for n in (T, T * k))
    w = torch.rand((T, k), device="cuda", generator=g)
    perm = torch.randperm(T * k, device="cuda", generator=g).int()
    bad = torch.rand(T * k, device="cuda", generator=g) < 0.3
    wild = torch.tensor([-2, -2 ** 31, T * k, 2 ** 31 - 1], dtype=torch.int64).to(torch.int32).cuda()
    announce("permuted indices out of range")
    res = []
    for p in (torch.where(bad, wild[torch.arange(T * k, device="cuda") % 4], perm), perm.masked_fill(bad, -1)):
        rows = torch.full((T * k, H), 5.0, dtype=torch.bfloat16, device="cuda")
        res.append(binding.finalize_backward(
            sh, d, y, {"expanded_idx_to_permuted_idx": p, "topk_weights": w}, d_expert_out=rows))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert (res[0][1].view(-1)[bad] == 0).all()
