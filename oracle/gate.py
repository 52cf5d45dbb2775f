"""The router in float64: top-K gate, load-balance loss, and the gradient of both.

Written from the definitions in include/moe_mx.h (moe_gate_topk, moe_balance_loss,
moe_gate_backward); no code shared with the kernels. The pages start at given
expert ids and gate weights (MegaMoE "Parameter Description", topk_ids and
topk_weights), so nothing on them pins these functions: the gradients are checked
against differences of the forward functions instead.

``*_magnitude`` outputs are the same expressions with every term taken by its absolute
value: the scale of the rounding errors of a 32-bit evaluation.
"""

from __future__ import annotations

import numpy as np


def clean(logits) -> np.ndarray:
    """float64 logits: NaN -> -inf, +inf -> the largest finite fp32 value."""
    x = np.asarray(logits, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    return np.minimum(x, float(np.finfo(np.float32).max))


def scores(logits, scoring: str) -> np.ndarray:
    x = clean(logits)
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    if x.shape[1] == 0 or x.shape[0] == 0:
        return np.zeros_like(x)
    m = x.max(axis=1, keepdims=True)
    e = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    total = e.sum(axis=1, keepdims=True)
    return e / np.where(total > 0, total, 1.0)


def topk(logits, k, scoring, bias=None, groups=1, topk_groups=1, renorm=True, scale=1.0):
    """(ids int32 [N, K], weights float64 [N, K])."""
    x = clean(logits)
    n, e = x.shape
    s = scores(logits, scoring)
    rank = x.copy() if bias is None else s + np.asarray(bias, np.float64)
    rank = np.where(np.isfinite(x) & ~np.isnan(rank), rank, -np.inf)
    ids = np.zeros((n, k), dtype=np.int32)
    w = np.zeros((n, k))
    for t in range(n):
        allowed = list(range(e))
        if groups > 1:
            size = e // groups
            best = []
            for g in range(groups):
                live = [s[t, i] if bias is None else rank[t, i] for i in range(g * size, (g + 1) * size)
                        if rank[t, i] > -np.inf]
                best.append(sum(sorted(live, reverse=True)[:2]) if live else -np.inf)
            keep = sorted(range(groups), key=lambda g: (-best[g], g))[:topk_groups]
            allowed = [i for i in range(e) if i // size in keep]
        order = sorted(allowed, key=lambda i: (-rank[t, i], i))[:k]
        ids[t] = order
        w[t] = [s[t, i] if np.isfinite(x[t, i]) else 0.0 for i in order]
    if renorm:
        total = w.sum(axis=1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    return ids, w * scale


def shares(logits, scoring):
    """p of the balance loss: the scores of a row over their sum."""
    s = scores(logits, scoring)
    if scoring == "sigmoid":
        z = s.sum(axis=1, keepdims=True)
        s = s / np.where(z > 0, z, 1.0)
    return s


def sequences(rows, offsets, mask):
    """Sequence of each row (-1: none, or not counted), number of sequences."""
    off = [0, rows] if offsets is None else [int(v) for v in offsets]
    seq = np.full(rows, -1)
    for b in range(len(off) - 1):
        seq[off[b]:off[b + 1]] = b
    if mask is not None:
        seq[np.asarray(mask) == 0] = -1
    return seq, len(off) - 1


def balance(logits, ids, scoring, offsets=None, mask=None, alpha=1.0):
    """(loss, counts int64 [B, E], coef [B, E])."""
    n, e = np.shape(logits)
    k = ids.shape[1]
    p = shares(logits, scoring)
    seq, seqs = sequences(n, offsets, mask)
    counts = np.zeros((seqs, e), dtype=np.int64)
    mean = np.zeros((seqs, e))
    held = np.zeros(seqs)
    for b in range(seqs):
        rows = seq == b
        held[b] = rows.sum()
        flat = ids[rows].reshape(-1)
        flat = flat[(flat >= 0) & (flat < e)]
        counts[b] = np.bincount(flat, minlength=e)[:e]
        if held[b]:
            mean[b] = p[rows].sum(axis=0) / held[b]
    filled = max(int((held > 0).sum()), 1)
    t = np.where(held > 0, held, 1.0)[:, None]
    share = e * counts / (k * t)
    loss = alpha / filled * float((share * mean).sum())
    return loss, counts, alpha * share / (t * filled)


def backward(logits, ids, scoring, grad_weights=None, renorm=True, scale=1.0, grad_loss=None, coef=None, offsets=None,
             mask=None):
    """(dlogits [N, E], its magnitude [N, E])."""
    n, e = np.shape(logits)
    s = scores(logits, scoring)
    d, dm = np.zeros((n, e)), np.zeros((n, e))
    if grad_weights is not None:
        sel = np.take_along_axis(s, ids, axis=1)
        g = np.asarray(grad_weights, np.float64) * scale
        gm = np.abs(g)
        if renorm:
            total = sel.sum(axis=1, keepdims=True)
            inv = np.where(total > 0, 1.0 / np.where(total > 0, total, 1.0), 0.0)
            gm = (gm + (gm * sel).sum(axis=1, keepdims=True) * inv) * inv
            g = (g - (g * sel).sum(axis=1, keepdims=True) * inv) * inv
        rows = np.arange(n)[:, None]
        np.add.at(d, (rows, ids), g)   # an id may stand in several places
        np.add.at(dm, (rows, ids), gm)
    q = np.zeros((n, e))
    if grad_loss is not None:
        seq, _ = sequences(n, offsets, mask)
        rows = seq >= 0
        q[rows] = float(np.reshape(grad_loss, -1)[0]) * np.asarray(coef, np.float64)[seq[rows]]
    if scoring == "softmax":
        d, dm = d + q, dm + np.abs(q)
        return (s * (d - (d * s).sum(axis=1, keepdims=True)),
                s * (dm + (dm * s).sum(axis=1, keepdims=True)))
    z = s.sum(axis=1, keepdims=True)
    inv = np.where(z > 0, 1.0 / np.where(z > 0, z, 1.0), 0.0)
    h = (q - (q * s).sum(axis=1, keepdims=True) * inv) * inv
    hm = (np.abs(q) + (np.abs(q) * s).sum(axis=1, keepdims=True) * inv) * inv
    return (d + h) * s * (1.0 - s), (dm + hm) * s * (1.0 - s)
