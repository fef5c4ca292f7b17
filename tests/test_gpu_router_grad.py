"""Balance loss, router gradient and finalize gradient on the GPU against their
formulas in float64, against differences, and together as a training step."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests import _router, _w4
from tests._gpu import announce, bf16_to_np

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24


def _shape(T, E, k, method=0, H=64, scaling=1.0):
    return binding.Shape(T, H, 32, E, k, 0, E, 0, 0, 0, scaling, 0, method)


def _offsets(rng, T, S, head=0, tail=0):
    """S ascending sequences of [head, T - tail), every third empty."""
    ends = np.sort(rng.integers(head, max(head, T - tail) + 1, S - 1)) if S > 1 else np.zeros(0, int)
    o = np.concatenate([[min(head, T)], ends, [max(head, T - tail)]])
    for i in range(2, S, 3):
        o[i] = o[i - 1]
    return np.minimum(np.maximum.accumulate(o), T).astype(np.int32)


# T, E, k, S, masked share, head and tail tokens outside every sequence
BALANCE = [
    (1, 1, 1, 1, 0.0, 0, 0), (1, 8, 2, 1, 0.0, 0, 0), (7, 64, 3, 1, 0.0, 0, 0),
    (64, 128, 8, 1, 0.0, 0, 0), (128, 65, 8, 16, 0.3, 0, 5), (129, 127, 8, 1, 0.5, 0, 0),
    (100, 256, 4, 17, 0.0, 3, 7), (333, 40, 6, 5, 0.2, 10, 33), (1000, 512, 8, 3, 0.1, 0, 1),
    (2048, 128, 8, 4, 0.0, 0, 0), (777, 1024, 64, 2, 0.1, 0, 0), (50, 300, 64, 1, 0.0, 0, 0),
    (20000, 60, 2, 40, 0.05, 100, 500), (300, 16, 2, 300, 0.0, 0, 0), (64, 32, 4, 2, 1.0, 0, 0),
]


def _tokens(rng, T, S, masked, head, tail):
    mask = (rng.random(T) >= masked).astype(np.uint8) if masked else None
    offsets = _offsets(rng, T, S, head, tail) if S > 1 or head or tail else None
    return mask, offsets


def _dev(a, dtype=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype)).cuda()


@pytest.mark.parametrize("T,E,k,S,masked,head,tail", BALANCE)
def test_balance_loss(T, E, k, S, masked, head, tail):
    """Counts and tokens exactly.  p errs by a few ulp (the exponential's and the
    quotient's 4, and E + log of fp32 sum steps of positive terms, of which each
    adds at most F32): relative (E + 16) F32; a mean over N <= T positive terms
    adds T F32 in any order; the loss adds E positive products on top."""
    rng = np.random.default_rng(T + E)
    mask, offsets = _tokens(rng, T, S, masked, head, tail)
    S = len(offsets) - 1 if offsets is not None else 1
    logits = (3 * rng.standard_normal((T, E))).astype(np.float32)
    ids = np.argsort(-logits, 1, kind="stable")[:, :k].astype(np.int32)
    seq, _ = _router.owner(T, mask, offsets)
    logits[seq < 0] = np.nan           # padding may hold anything
    ids[seq < 0] = -7
    announce(f"balance_loss T={T} E={E} k={k} S={S}")
    r = binding.balance_loss(_shape(T, E, k), _dev(logits), _dev(ids), _dev(mask), _dev(offsets))
    torch.cuda.synchronize()
    loss, counts, probs, tokens, _ = _router.balance(logits, ids, seq, S)
    np.testing.assert_array_equal(r["counts"].cpu().numpy(), counts)
    np.testing.assert_array_equal(r["tokens"].cpu().numpy(), tokens)
    # the exponential's argument x - max is rounded: up to |x - max| F32 more
    span = np.nanmax(logits[seq >= 0], initial=0) - np.nanmin(logits[seq >= 0], initial=0)
    rel = (E + T + 16 + 2 * span) * F32
    assert (np.abs(r["probs"].cpu().numpy() - probs) <= rel * probs).all()
    assert abs(float(r["loss"]) - loss) <= (rel + (E + S + 8) * F32) * loss


@pytest.mark.parametrize("method", [0, 1])
@pytest.mark.parametrize("with_weights,with_balance", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("T,E,k,S,masked,head,tail", BALANCE[:9] + BALANCE[10:12] + BALANCE[13:])
def test_route_backward(T, E, k, S, masked, head, tail, with_weights, with_balance, method):
    """Each term of a row errs by a few relative roundings of its factors: p by
    (E + 16 + 2 span) F32, sums over k slots by k F32 and over E by E F32 of their
    absolute terms."""
    rng = np.random.default_rng(T * 3 + E + method)
    mask, offsets = _tokens(rng, T, S, masked, head, tail)
    S = len(offsets) - 1 if offsets is not None else 1
    logits = (2 * rng.standard_normal((T, E))).astype(np.float32)
    c = _w4.W4Case("route", T, 64, 32, E, k, method=method)
    ids, w = _w4.route(c, logits)
    ids, w = ids.astype(np.int32), w.astype(np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    seq, _ = _router.owner(T, mask, offsets)
    _, counts, _, tokens, _ = _router.balance(logits, ids, seq, S)
    for a in (logits, w, dw):
        a[seq < 0] = np.nan
    announce(f"route_backward T={T} E={E} k={k} S={S} method={method} {with_weights} {with_balance}")
    d_loss = 0.37
    kept = {"counts": _dev(counts, np.int32), "tokens": _dev(tokens, np.int32)}
    out = torch.full((T, E), float("nan"), device="cuda")
    got = binding.route_backward(
        _shape(T, E, k, method), _dev(logits), _dev(ids), _dev(w),
        d_topk_weights=_dev(dw) if with_weights else None, balance=kept if with_balance else None,
        d_loss=torch.full((1,), d_loss, device="cuda") if with_balance else None,
        token_mask=_dev(mask), seq_offsets=_dev(offsets), d_logits=out)
    assert got.data_ptr() == out.data_ptr()
    got = got.cpu().numpy()
    args = dict(w=w if with_weights else None, dw=dw if with_weights else None, method=method,
                d_loss=float(np.float32(d_loss)) if with_balance else None, counts=counts, tokens=tokens)
    want = _router.logits_gradient(logits, ids, seq, S, **args)
    assert (got[seq < 0] == 0).all()
    span = np.nanmax(logits[seq >= 0], initial=0) - np.nanmin(logits[seq >= 0], initial=0)
    rel = (2 * E + 2 * k + 40 + 2 * span) * F32
    size = np.zeros((T, E))            # the absolute terms that a row's entries are made of
    used = max(1, int((tokens > 0).sum()))
    for t in np.flatnonzero(seq >= 0):
        p = _router.softmax(logits[t:t + 1])[0]
        if with_weights:
            inside = np.abs(w[t].astype(np.float64) * dw[t]).sum()
            for j in range(k):
                size[t, ids[t, j]] += w[t, j] * (abs(dw[t, j]) + inside)
            size[t] += p * inside
        if with_balance:
            g = d_loss * E * counts[seq[t]] / (k * float(tokens[seq[t]]) ** 2 * used)
            size[t] += p * (g + (p * g).sum())
    assert (np.abs(got - want) <= rel * size).all()


@pytest.mark.parametrize("T,E,k,S", [(70000, 5, 2, 65535), (300000, 16, 3, 7)])
def test_many_sequences_and_tokens(T, E, k, S):
    """As many sequences as there may be, a third of them empty, and long ones
    over many chunks; bounds as above with the longest sequence's N."""
    rng = np.random.default_rng(S)
    mask, offsets = (rng.random(T) >= 0.1).astype(np.uint8), _offsets(rng, T, S, 3, 9)
    x = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(-x, 1, kind="stable")[:, :k].astype(np.int32)
    announce(f"balance_loss, route_backward T={T} S={S}")
    sh = _shape(T, E, k)
    r = binding.balance_loss(sh, _dev(x), _dev(ids), _dev(mask), _dev(offsets))
    got = binding.route_backward(sh, _dev(x), balance=r, d_loss=torch.ones(1, device="cuda"),
                                 token_mask=_dev(mask), seq_offsets=_dev(offsets)).cpu().numpy()
    seq = np.searchsorted(offsets, np.arange(T), "right") - 1
    seq = np.where((mask != 0) & (seq >= 0) & (seq < S), seq, -1)
    live = seq >= 0
    p = _router.softmax(x)
    counts, total = np.zeros((S, E)), np.zeros((S, E))
    tokens = np.bincount(seq[live], minlength=S)
    np.add.at(counts, (np.repeat(seq[live], k), ids[live].reshape(-1)), 1)
    np.add.at(total, seq[live], p[live])
    inv = 1 / np.maximum(tokens, 1)[:, None]
    probs = total * inv
    loss = (E / k * inv * counts * probs).sum() / (tokens > 0).sum()
    np.testing.assert_array_equal(r["counts"].cpu().numpy(), counts)
    np.testing.assert_array_equal(r["tokens"].cpu().numpy(), tokens)
    rel = (E + tokens.max() + 16 + 2 * (x.max() - x.min())) * F32
    assert (np.abs(r["probs"].cpu().numpy() - probs) <= rel * probs).all()
    assert abs(float(r["loss"]) - loss) <= (rel + (E + S + 8) * F32) * loss
    g = E / k * inv ** 2 * counts / (tokens > 0).sum()
    g = np.where(live[:, None], g[seq], 0)
    inner = (p * g).sum(1, keepdims=True)
    rel = (2 * E + 2 * k + 40 + 2 * (x.max() - x.min())) * F32
    assert (np.abs(got - p * (g - inner)) <= rel * p * (g + inner)).all()
    assert (got[~live] == 0).all()


def test_empty_rows_and_extreme_logits():
    """Experts masked by -inf or by the type's lowest value, a row of -inf only
    (no distribution: probabilities and gradient 0), huge logits."""
    T, E, k = 6, 8, 2
    low = np.finfo(np.float32).min
    rng = np.random.default_rng(0)
    x = rng.standard_normal((T, E)).astype(np.float32)
    x[0] = -np.inf
    x[1, 2:] = -np.inf
    x[2] = low
    x[3, 3:] = low
    x[4] = 3e38
    ids = np.tile(np.array([0, 1], np.int32), (T, 1))
    w = np.full((T, k), 0.5, np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    announce("extreme logits")
    sh = _shape(T, E, k, 1)
    r = binding.balance_loss(sh, _dev(x), _dev(ids))
    got = binding.route_backward(sh, _dev(x), _dev(ids), _dev(w), _dev(dw), balance=r,
                                 d_loss=torch.ones(1, device="cuda")).cpu().numpy()
    seq, S = _router.owner(T)
    loss, counts, probs, tokens, _ = _router.balance(x, ids, seq, S)
    np.testing.assert_array_equal(r["counts"].cpu().numpy(), counts)
    np.testing.assert_allclose(r["probs"].cpu().numpy(), probs, rtol=64 * F32)
    np.testing.assert_allclose(float(r["loss"]), loss, rtol=64 * F32)
    want = _router.logits_gradient(x, ids, seq, S, w, dw, 1, 1.0, counts, tokens)
    np.testing.assert_allclose(got, want, rtol=0, atol=200 * F32)
    assert np.isfinite(got).all() and (got[0, 2:] == 0).all()


def test_repeated_and_foreign_ids():
    """The same id several times in one token, and ids of no expert: one sum for
    the expert, nothing for the others, the same bits in every run."""
    T, E, k = 40, 12, 6
    rng = np.random.default_rng(2)
    ids = rng.integers(-2, E + 2, (T, k)).astype(np.int32)
    ids[0], ids[1], ids[2, :4] = 3, -1, 5
    x = rng.standard_normal((T, E)).astype(np.float32)
    w, dw = (rng.standard_normal((T, k)).astype(np.float32) for _ in range(2))
    announce("repeated ids")
    seq, S = _router.owner(T)
    for method in (0, 1):
        sh = _shape(T, E, k, method)
        r = binding.balance_loss(sh, _dev(x), _dev(ids))
        _, counts, _, tokens, _ = _router.balance(x, ids, seq, S)
        np.testing.assert_array_equal(r["counts"].cpu().numpy(), counts)
        runs = [binding.route_backward(sh, _dev(x), _dev(ids), _dev(w), _dev(dw)).cpu().numpy()
                for _ in range(3)]
        want = _router.logits_gradient(x, ids, seq, S, w, dw, method)
        size = (np.abs(w) * (np.abs(dw) + np.abs(w * dw).sum(1, keepdims=True))).sum(1)
        assert (np.abs(runs[0] - want) <= (2 * E + 4 * k + 40) * F32 * size[:, None]).all()
        assert all((q == runs[0]).all() for q in runs)


def test_gradient_against_differences():
    """Central differences of the float64 loss; the counts stay as they are."""
    T, E, k, S = 12, 10, 3, 2
    rng = np.random.default_rng(11)
    x = rng.standard_normal((T, E)).astype(np.float32)
    offsets = np.array([0, 5, 12], np.int32)
    seq, _ = _router.owner(T, None, offsets)
    v = rng.standard_normal((T, k))
    announce("differences")
    for method in (0, 1):
        c = _w4.W4Case("diff", T, 64, 32, E, k, method=method)
        ids, w = _w4.route(c, x)

        def f(z):
            p = _router.softmax(z)
            _, counts, _, tokens, _ = _router.balance(x, ids, seq, S)
            total = 0.0
            for s in range(S):
                total += E / (k * tokens[s]) * (counts[s] * p[seq == s].mean(0)).sum() / S
            top = np.take_along_axis(z, ids, 1)
            e = np.exp(top)
            wz = e / (np.exp(z).sum(1, keepdims=True) if method else e.sum(1, keepdims=True))
            return 0.5 * total + (wz * v).sum()

        h, want = 1e-5, np.zeros((T, E))
        z = x.astype(np.float64)
        for t in range(T):
            for e in range(E):
                up, down = z.copy(), z.copy()
                up[t, e] += h
                down[t, e] -= h
                want[t, e] = (f(up) - f(down)) / (2 * h)
        sh = _shape(T, E, k, method)
        ids = ids.astype(np.int32)
        r = binding.balance_loss(sh, _dev(x), _dev(ids), seq_offsets=_dev(offsets))
        got = binding.route_backward(sh, _dev(x), _dev(ids), _dev(w, np.float32), _dev(v, np.float32),
                                     balance=r, d_loss=torch.full((1,), 0.5, device="cuda"),
                                     seq_offsets=_dev(offsets)).cpu().numpy()
        # the differences: h^2 times a third derivative of order 1, 2^-52 |f| / h; the
        # kernel: (2 E + 2 k + 40 + 2 span) F32 of terms that add up to less than 1
        assert np.abs(got - want).max() <= 1e-8 + (2 * E + 2 * k + 60) * F32


@pytest.mark.parametrize("T,H,k,local,scaling", [
    (1, 64, 1, 1.0, 1.0), (3, 64, 5, 0.0, 1.0), (16, 2048, 8, 1.0, 2.5), (33, 1088, 6, 0.4, 1.0),
    (5, 4160, 3, 0.7, 0.5), (200, 512, 8, 0.3, 1.0)])
def test_finalize_backward(T, H, k, local, scaling):
    rng = np.random.default_rng(T + H)
    n = T * k
    here = rng.random(n) < local
    perm = np.full(n, -1, np.int32)
    perm[here] = rng.permutation(int(here.sum()))
    d, y = _w4.bf16(rng.standard_normal((T, H))), _w4.bf16(rng.standard_normal((n, H)))
    y[int(here.sum()):] = np.nan                       # rows of no slot
    w = rng.random((T, k)).astype(np.float32)
    sh = _shape(T, 64, k, 0, H, scaling)
    r = {"expanded_idx_to_permuted_idx": _dev(perm), "topk_weights": _dev(w)}
    rows = torch.full((n, H), 9.0, dtype=torch.bfloat16, device="cuda")
    announce(f"finalize_backward T={T} H={H} k={k}")
    dy, dw = binding.finalize_backward(sh, _dev(d).bfloat16(), _dev(y).bfloat16(), r, d_expert_out=rows)
    only_w = binding.finalize_backward(sh, _dev(d).bfloat16(), _dev(y).bfloat16(), r, expert_out_grad=False)
    only_y = binding.finalize_backward(sh, _dev(d).bfloat16(), None, r, weights_grad=False)
    assert only_w[0] is None and only_y[1] is None
    assert torch.equal(only_w[1], dw)
    dy, dw = bf16_to_np(dy), dw.cpu().numpy()
    P = int(here.sum())
    assert (dy[P:] == 9.0).all()
    assert (bf16_to_np(only_y[0])[:P] == dy[:P]).all()
    for x in range(n):
        t, j, p = x // k, x % k, perm[x]
        if p < 0:
            assert dw[t, j] == 0
            continue
        want = np.float64(scaling) * w[t, j] * d[t]
        assert (np.abs(dy[p] - want) <= (_w4.U + 4 * F32) * np.abs(want)).all()
        terms = d[t].astype(np.float64) * y[p]
        assert abs(dw[t, j] - scaling * terms.sum()) <= scaling * (H + 4) * F32 * np.abs(terms).sum()


def test_gradients_in_place():
    """d_logits over router_logits and d_expert_out over expert_out: the same bits."""
    T, E, k, H = 700, 96, 5, 320
    rng = np.random.default_rng(21)
    sh = _shape(T, E, k, 1, H)
    x = _dev(rng.standard_normal((T, E)), np.float32)
    ids = _dev(np.argsort(-x.cpu().numpy(), 1, kind="stable")[:, :k], np.int32)
    w, dw = (_dev(rng.standard_normal((T, k)), np.float32) for _ in range(2))
    one = torch.ones(1, device="cuda")
    announce("in place")
    bal = binding.balance_loss(sh, x, ids)
    want = binding.route_backward(sh, x, ids, w, dw, balance=bal, d_loss=one)
    here = x.clone()
    binding.route_backward(sh, here, ids, w, dw, balance=bal, d_loss=one, d_logits=here)
    assert torch.equal(here, want)
    d, y = (_dev(rng.standard_normal((n, H)), np.float32).bfloat16() for n in (T, T * k))
    r = {"expanded_idx_to_permuted_idx": _dev(rng.permutation(T * k), np.int32), "topk_weights": w}
    dy, dw_want = binding.finalize_backward(sh, d, y, r)
    _, dw_here = binding.finalize_backward(sh, d, y, r, d_expert_out=y)
    assert torch.equal(y, dy) and torch.equal(dw_here, dw_want)


def test_two_streams_at_once():
    """Steps of different sizes on two streams, each with workspaces of its own."""
    steps, want = [], []
    for seed, T, E in ((1, 1500, 128), (2, 40, 64)):
        c = _w4.W4Case("stream", T, 192, 96, E, 4, L=2, rg=8, rd=8, zeros=1, group=64, seed=seed)
        x = _w4.inputs(c)
        shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
        r = binding.alloc_routing(shape, "cuda")

        def step(shape=shape, fmt=fmt, hidden=hidden, packed=packed, kw=kw, logits=logits, r=r):
            out = binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, routing=r, **kw)
            bal = binding.balance_loss(shape, logits, r["topk_ids"])
            d = binding.route_backward(shape, logits, balance=bal,
                                       d_loss=torch.ones(1, device="cuda"))
            return out, bal["loss"], d

        steps.append(step)
        want.append([t.clone() for t in step()])
    announce("two streams")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [[], []]
    for _ in range(8):
        for i, (s, step) in enumerate(zip(streams, steps)):
            with torch.cuda.stream(s):
                got[i].append(step())
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, w))


def test_training_step_together():
    """forward_w4 with its expert outputs -> finalize -> balance loss -> the
    gradient of the router's logits, against the chain in float64."""
    c = _w4.W4Case("train", 48, 192, 96, 10, 3, L=2, rg=8, rd=8, zeros=1, group=64, method=1, scaling=1.5)
    x = _w4.inputs(c)
    shape, fmt, hidden, packed, kw, logits = _w4.device_layer(c, x)
    rng = np.random.default_rng(8)
    mask = (rng.random(c.T) > 0.2).astype(np.uint8)
    offsets = np.array([0, 20, 20, 44], np.int32)
    d_out = _w4.bf16(rng.standard_normal((c.T, c.H)))
    announce("training step")
    rows = torch.empty((c.T * c.k, c.H), dtype=torch.bfloat16, device="cuda")
    r = binding.alloc_routing(shape, "cuda")
    binding.forward_w4(shape, fmt, hidden, *packed, router_logits=logits, routing=r, expert_out=rows, **kw)
    binding.finalize(shape, rows, r)
    bal = binding.balance_loss(shape, logits, r["topk_ids"], _dev(mask), _dev(offsets))
    _, dw = binding.finalize_backward(shape, _dev(d_out).bfloat16(), rows, r, expert_out_grad=False)
    d = binding.route_backward(shape, logits, r["topk_ids"], r["topk_weights"], dw, balance=bal,
                               d_loss=torch.full((1,), 0.01, device="cuda"), token_mask=_dev(mask),
                               seq_offsets=_dev(offsets)).cpu().numpy()
    ids, w = _w4.route(c, x["logits"])
    np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), ids)
    _, _, slots = _w4.reference(c, x)
    seq, S = _router.owner(c.T, mask, offsets)
    loss, counts, _, tokens, _ = _router.balance(x["logits"], ids, seq, S)
    assert abs(float(bal["loss"]) - loss) <= 1e-5 * loss
    dw_want, dw_off = np.zeros((c.T, c.k)), np.zeros((c.T, c.k))
    for (t, j), y in slots.items():
        one = np.full((c.T, c.k), -1)
        one[t, j] = ids[t, j]
        dw_want[t, j] = c.scaling * (d_out[t].astype(np.float64) * y).sum()
    got_dw = dw.cpu().numpy()
    # the rows err by the layer's three bf16 roundings: 2-norms, relative to |d_out| |y|
    for (t, j), y in slots.items():
        dw_off[t, j] = c.scaling * 3 * _w4.U * np.linalg.norm(d_out[t]) * np.linalg.norm(y)
        assert abs(got_dw[t, j] - dw_want[t, j]) <= dw_off[t, j]
    want = _router.logits_gradient(x["logits"], ids, seq, S, w, got_dw, c.method,
                                   float(np.float32(0.01)), counts, tokens)
    size = np.abs(w * got_dw).sum(1, keepdims=True) + 0.01 * c.E
    assert (np.abs(d - want) <= 200 * F32 * size).all()
    assert (d[seq < 0] == 0).all()


def test_backward_graph_replays():
    """The step captured once and replayed with eager work between."""
    T, E, k = 200, 64, 4
    rng = np.random.default_rng(1)
    x = _dev(rng.standard_normal((T, E)), np.float32)
    ids = _dev(np.argsort(-x.cpu().numpy(), 1, kind="stable")[:, :k], np.int32)
    w = torch.full((T, k), 0.25, device="cuda")
    dw = _dev(rng.standard_normal((T, k)), np.float32)
    one = torch.ones(1, device="cuda")
    sh = _shape(T, E, k, 1)
    announce("router graph")

    def step():
        bal = binding.balance_loss(sh, x, ids)
        return bal, binding.route_backward(sh, x, ids, w, dw, balance=bal, d_loss=one)

    bal, d = step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bal_g, d_g = step()
    for _ in range(3):
        d_g.fill_(float("nan"))
        bal_g["loss"].fill_(float("nan"))
        g.replay()
        again = step()
        torch.cuda.synchronize()
        assert torch.equal(d_g, d) and torch.equal(again[1], d)
        for name in bal:
            assert torch.equal(bal_g[name], bal[name]) and torch.equal(again[0][name], bal[name])
