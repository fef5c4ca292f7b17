"""The balance loss and the router's and finalize's gradients in float64, from
their formulas (numpy)."""
import numpy as np


def owner(T, mask=None, offsets=None):
    """Sequence of each token (-1: takes no part) and the number of sequences."""
    seq, S = np.zeros(T, int), 1
    if offsets is not None:
        S = len(offsets) - 1
        seq[:] = -1
        for s in range(S):
            seq[offsets[s]:offsets[s + 1]] = s
    if mask is not None:
        seq = np.where(np.asarray(mask) != 0, seq, -1)
    return seq, S


def softmax(x):
    x = np.asarray(x, np.float64)
    top = np.where(np.isneginf(x.max(1, keepdims=True)), 0, x.max(1, keepdims=True))
    e = np.exp(x - top)
    total = e.sum(1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def balance(logits, ids, seq, S):
    """loss, counts, probs, tokens and p, over tokens with seq >= 0 only."""
    T, E = logits.shape
    k = ids.shape[1]
    p = np.zeros((T, E))
    live = seq >= 0
    if live.any():
        p[live] = softmax(logits[live])
    counts, probs, tokens = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros(S, np.int64)
    losses = []
    for s in range(S):
        rows = np.flatnonzero(seq == s)
        tokens[s] = len(rows)
        for e in ids[rows].reshape(-1):
            if 0 <= e < E:
                counts[s, e] += 1
        if len(rows):
            probs[s] = p[rows].mean(0)
            losses.append(E / (k * len(rows)) * (counts[s] * probs[s]).sum())
    return (float(np.mean(losses)) if losses else 0.0), counts, probs, tokens, p


def logits_gradient(logits, ids, seq, S, w=None, dw=None, method=0, d_loss=None, counts=None,
                    tokens=None):
    T, E = logits.shape
    k = ids.shape[1]
    d = np.zeros((T, E))
    used = max(1, int((tokens > 0).sum())) if tokens is not None else 1
    for t in range(T):
        if seq[t] < 0:
            continue
        p = softmax(logits[t:t + 1])[0]
        if dw is not None:
            ok = [j for j in range(k) if 0 <= ids[t, j] < E]
            inside = sum(float(w[t, j]) * float(dw[t, j]) for j in ok)
            for j in ok:
                d[t, ids[t, j]] += float(w[t, j]) * (float(dw[t, j]) - (inside if method == 0 else 0))
            if method == 1:
                d[t] -= p * inside
        if d_loss is not None:
            s = seq[t]
            g = d_loss * E * counts[s] / (k * float(tokens[s]) ** 2 * used)
            d[t] += p * (g - (p * g).sum())
    return d
