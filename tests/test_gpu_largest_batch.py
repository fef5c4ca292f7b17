"""The largest batch that a shape may have: 2^24 tokens of one slot each."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _w4
from tests._gpu import announce, bf16_to_np
from tests._w4 import W4Case
from tests.test_gpu_w4_blocks import _reference

pytestmark = pytest.mark.gpu

T = 1 << 24


def test_forward_w4():
    """Rows at both ends, in the middle and at random, against the definition."""
    c = W4Case("largest", T, 64, 32, 1, 1, group=64, zeros=1)
    few = W4Case("few", 4096, 64, 32, 1, 1, group=64, zeros=1)
    x = _w4.inputs(few)
    announce("forward_w4 2^24 tokens")
    _, fmt, _, packed, _, _ = _w4.device_layer(few, x)
    g = torch.Generator("cuda").manual_seed(2)
    hidden = torch.empty((T, c.H), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    out = torch.full((T, c.H), float("nan"), dtype=torch.bfloat16, device="cuda")
    binding.forward_w4(c.shape(), fmt, hidden, *packed, router_logits=torch.zeros((T, 1), device="cuda"), out=out)
    rng = np.random.default_rng(0)
    at = np.concatenate([np.arange(1024), T // 2 + np.arange(-512, 512), T - 1 - np.arange(1024),
                         rng.integers(0, T, 1024)])
    rows = torch.from_numpy(at).cuda()
    x["hidden"], x["logits"] = bf16_to_np(hidden[rows]).astype(np.float32), np.zeros((4096, 1), np.float32)
    ref, bound = _reference(few, x)
    assert (np.abs(bf16_to_np(out[rows]) - ref) <= bound).all()
    assert not out.isnan().any()


def test_finalize_and_its_gradients():
    """One slot a token, in reverse order: a copy of rows times an exact weight."""
    sh = binding.Shape(T, 64, 32, 1, 1, 0, 1, 0, 0, 0, 1.0, 0, 0)
    announce("finalize 2^24 tokens")
    y = torch.empty((T, 64), dtype=torch.bfloat16, device="cuda").normal_()
    r = {"expanded_idx_to_permuted_idx": torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda"),
         "topk_weights": torch.full((T, 1), 0.5, device="cuda")}
    out = torch.full_like(y, float("nan"))
    binding.finalize(sh, y, r, out=out)
    assert torch.equal(out, (y * 0.5).flip(0))
    d_y, d_w = binding.finalize_backward(sh, out, y, r)
    assert torch.equal(d_y, (out * 0.5).flip(0))
    # a sum of 64 products that are all half a square
    want = (y.float() ** 2).sum(1).flip(0)[:, None] * 0.5
    assert ((d_w - want).abs() <= 2 * 68 * 2.0 ** -24 * want).all()


def test_router():
    """Two experts: p = 1 / (1 + exp(difference)).  The sums over 2^24 positive terms
    run in chains of at most 4096 + 8 + 64 terms, each rounding relative to it."""
    E, k = 2, 1
    sh = binding.Shape(T, 64, 32, E, k, 0, E, 0, 0, 0, 1.0, 0, 0)
    announce("balance_loss, route_backward 2^24 tokens")
    x = torch.empty((T, E), device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    ids = x.argmax(1, keepdim=True).int()
    bal = binding.balance_loss(sh, x, ids)
    d = binding.route_backward(sh, x, balance=bal, d_loss=torch.ones(1, device="cuda"))
    p = torch.softmax(x.double(), 1)
    n = torch.bincount(ids.view(-1).long(), minlength=E)
    assert torch.equal(bal["counts"][0].long(), n) and int(bal["tokens"]) == T
    rel = (4096 + 8 + 64 + 32) * 2.0 ** -24
    assert ((bal["probs"][0] - p.mean(0)).abs() <= rel * p.mean(0)).all()
    loss = float(E * (n.double() / T * p.mean(0)).sum())
    assert abs(float(bal["loss"]) - loss) <= (rel + 16 * 2.0 ** -24) * loss
    g = E * n.double() / float(T) ** 2
    size = p * (g + (p * g).sum(1, keepdim=True))
    # as for small batches: (2 E + 2 k + 40 + 2 span) roundings of the absolute terms
    assert ((d - p * (g - (p * g).sum(1, keepdim=True))).abs() <= 80 * 2.0 ** -24 * size).all()
