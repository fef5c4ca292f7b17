"""The 4-bit layer with infinities and NaN: they stay in the tokens they belong
to, every other token keeps its bits."""
import dataclasses

import numpy as np
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _w4
from tests._gpu import announce, bf16_to_np
from tests._w4 import W4Case

pytestmark = pytest.mark.gpu

# tiles of 16, 32 and 64 rows; whole and odd ranks, several rank steps, one stack
# per adapter, several shares of K (one token)
CASES = [
    W4Case("rows16", 40, 128, 64, 8, 2, L=3, rg=8, rd=16, zeros=1, group=64),
    W4Case("rows16_odd_ranks", 44, 192, 96, 8, 2, L=3, rg=13, rd=37, shared=1),
    W4Case("rows16_k_shares", 6, 2048, 768, 6, 2, L=2, rg=16, rd=8),
    W4Case("rows32", 400, 128, 64, 2, 1, L=3, rg=40, rd=8, group=32),
    W4Case("rows32_adapters64", 400, 64, 32, 2, 1, L=64, rg=8, rd=5, zeros=1),
    W4Case("rows64", 4100, 128, 64, 3, 1, L=3, rg=16, rd=64),
]
BAD = 1  # the adapter with the bad values


def _outputs(c, x):
    shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
    out = binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, **kw)
    torch.cuda.synchronize()
    return bf16_to_np(out)


def _inputs(c):
    x = _w4.inputs(c)
    x["mapping"][:4] = (BAD, -1, 0, BAD)  # a tile with the adapter, without one, with another
    return x


@pytest.mark.parametrize("value", [np.inf, np.nan])
@pytest.mark.parametrize("where", ["b_gu", "b_dn", "a_gu", "a_dn"])
@pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
def test_bad_adapter_stays_with_its_tokens(c, where, value):
    x = _inputs(c)
    announce(f"{where} {value} {c}")
    clean = _outputs(c, x)
    hit = x[where][BAD]                         # every expert's stack of the adapter
    saved = hit.copy()
    hit[:, 4, hit.shape[2] - 1] = value         # the last rank position (b) or K column (a)
    got = _outputs(c, x)
    own = x["mapping"] == BAD
    assert (got[~own] == clean[~own]).all()
    if where != "b_dn":
        assert (~np.isfinite(got[own])).any(1).all()
        return
    # one column of the output; the others hold to the definition
    assert not np.isfinite(got[own, 4]).any()
    hit[:] = saved
    n = min(c.T, 24)
    ref, bound, _ = _w4.reference(dataclasses.replace(c, T=n), {**x, "logits": x["logits"][:n]})
    over = np.abs(got[:n] - ref)[own[:n]] > bound[own[:n]]
    assert not np.delete(over, 4, 1).any()


@pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
def test_bad_hidden_rows_stay_alone(c):
    x = _inputs(c)
    announce(f"hidden {c}")
    clean = _outputs(c, x)
    x["hidden"][0, 3], x["hidden"][3, c.H - 1], x["hidden"][4, 40] = np.nan, np.inf, -np.inf
    got = _outputs(c, x)
    bad = np.isin(np.arange(c.T), (0, 3, 4))
    assert not np.isfinite(got[bad]).any()
    assert (got[~bad] == clean[~bad]).all()
