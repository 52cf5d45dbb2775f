"""The norm and the 16-bit products of expert groups in float64, with their gradients.

Written from the definitions in include/moe_mx.h (moe_rms_norm, moe_rms_norm_backward,
moe_grouped_matmul, moe_grouped_matmul_wgrad); no code shared with the kernels. None of
the pages defines them; the gradients are checked against differences of the forward
functions. Parity unpinned.
"""

from __future__ import annotations

import numpy as np


def rms_norm(h, weight, eps):
    """(y, rstd) of the rows h as they are kept."""
    h = np.asarray(h, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * np.asarray(weight, np.float64), rstd


def rms_norm_backward(grad_y, h, weight, rstd, grad_h=None):
    """(grad_x, grad_weight) for rows whose rstd is that of their norm."""
    g, h = np.asarray(grad_y, np.float64), np.asarray(h, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    xh, a = h * r, g * np.asarray(weight, np.float64)
    gx = r * (a - xh * (a * xh).sum(axis=1, keepdims=True) / h.shape[1])
    if grad_h is not None:
        gx = gx + np.asarray(grad_h, np.float64)
    return gx, (g * xh).sum(axis=0)


def groups(offsets, rows):
    return [(0, rows)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def grouped_matmul(x, w, offsets=None, transpose_w=False):
    """(out, magnitude): the product and that of the absolute values; NaN where no group is."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    n = w.shape[2] if transpose_w else w.shape[1]
    out, mag = np.full((x.shape[0], n), np.nan), np.full((x.shape[0], n), np.nan)
    for g, (lo, hi) in enumerate(groups(offsets, x.shape[0])):
        m = w[g] if transpose_w else w[g].T
        out[lo:hi], mag[lo:hi] = x[lo:hi] @ m, np.abs(x[lo:hi]) @ np.abs(m)
    return out, mag


def grouped_matmul_wgrad(grad_out, x, offsets=None):
    """(grad_w [G, N, K], magnitude)."""
    g, x = np.asarray(grad_out, np.float64), np.asarray(x, np.float64)
    out, mag = [], []
    for lo, hi in groups(offsets, x.shape[0]):
        out.append(g[lo:hi].T @ x[lo:hi])
        mag.append(np.abs(g[lo:hi]).T @ np.abs(x[lo:hi]))
    return np.stack(out), np.stack(mag)
