"""The balance loss on both sides of the sizes where one block does a whole
batch (no workspace) and where two launches do."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _router
from tests._gpu import announce

F32 = 2.0 ** -24

# T, E, k, S, one block: by time, one block walks sequence after sequence
PATHS = [
    (32, 128, 8, 16, True), (32, 64, 4, 17, False), (33, 128, 8, 7, True), (33, 128, 8, 8, False),
    (64, 256, 8, 4, True), (64, 256, 8, 5, False), (64, 257, 8, 1, False), (128, 128, 8, 2, True),
    (128, 128, 8, 3, False), (128, 129, 8, 1, False), (129, 64, 2, 1, False), (128, 128, 8, 16, False),
    (64, 128, 8, 16, False), (16, 1024, 8, 16, True), (5, 12, 3, 9, True),
]


def _size(T, E, k, S):
    sh = binding.Shape(T, 64, 32, E, k, 0, E, 0, 0, 0, 1.0, 0, 0)
    return sh, binding.load_library().moe_lora_balance_workspace_size(sh, S)


@pytest.mark.parametrize("T,E,k,S,one", PATHS)
def test_workspace_goes_by_the_faster_side(T, E, k, S, one):
    assert (_size(T, E, k, S)[1] == 0) == one


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,S,one", PATHS)
def test_balance_loss_on_both_sides(T, E, k, S, one):
    """Bounds as in test_gpu_router_grad.py: (E + T + 16 + 2 span) F32 for the mean
    probabilities, E + S + 8 more for the loss."""
    rng = np.random.default_rng(T * S)
    sh, size = _size(T, E, k, S)
    offsets = np.sort(np.concatenate([[0, T], rng.integers(0, T + 1, S - 1)])).astype(np.int32)
    mask = (rng.random(T) >= 0.2).astype(np.uint8)
    x = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(-x, 1, kind="stable")[:, :k].astype(np.int32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    announce(f"balance_loss T={T} E={E} S={S} workspace {size}")
    r = binding.balance_loss(sh, dev(x), dev(ids), dev(mask), dev(offsets))
    seq, _ = _router.owner(T, mask, offsets)
    loss, counts, probs, tokens, _ = _router.balance(x, ids, seq, S)
    np.testing.assert_array_equal(r["counts"].cpu().numpy(), counts)
    np.testing.assert_array_equal(r["tokens"].cpu().numpy(), tokens)
    rel = (E + T + 16 + 2 * (x.max() - x.min())) * F32
    assert (np.abs(r["probs"].cpu().numpy() - probs) <= rel * probs).all()
    assert abs(float(r["loss"]) - loss) <= (rel + (E + S + 8) * F32) * loss
