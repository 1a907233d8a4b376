"""Plain fp64 CPU oracle of the operators around the output head.

TEST INFRASTRUCTURE ONLY (see kl_oracle.py).  Layer norm and its gradients,
8-bit activation checkpoints, head logits and token sampling, each from its
definition; it shares no code with the HIP library.

8-bit checkpoints are defined by single-precision steps (per row and block of
128: scale = max(amax * fl(1/127), 2^-126), q = clamp(rint(x * fl(1/scale)),
+-127)), so their bytes and scales are compared exactly; the values they stand
for are q * scale in float64.
"""
from __future__ import annotations

import numpy as np

__all__ = ["layer_norm", "layer_norm_grads", "act8", "act8_values", "sample"]

BLOCK = 128


def layer_norm(x, weight, bias, eps):
    """(y, mean, rstd) in float64; bias may be None."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def layer_norm_grads(dy, x, weight, mean, rstd):
    """(dx, dweight, dbias) in float64, with the given statistics."""
    dy, x, w = (np.asarray(a, np.float64) for a in (dy, x, weight))
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def act8(x):
    """(q int8 [T, d], scale float32 [T, blocks]) of float32 x [T, d]."""
    x = np.asarray(x, np.float32)
    T, d = x.shape
    q = np.zeros((T, d), np.int8)
    scale = np.empty((T, -(-d // BLOCK)), np.float32)
    for j in range(scale.shape[1]):
        b = x[:, j * BLOCK:(j + 1) * BLOCK]
        good = np.isfinite(b).all(1)
        amax = np.where(good, np.abs(np.where(good[:, None], b, 0)).max(1), np.float32(0)).astype(np.float32)
        s = np.maximum(amax * (np.float32(1) / np.float32(127)), np.float32(2.0 ** -126))
        v = np.where(good[:, None], b, np.float32(0)) * (np.float32(1) / s)[:, None]
        q[:, j * BLOCK:(j + 1) * BLOCK] = np.clip(np.rint(v), -127, 127)
        scale[:, j] = np.where(good, s, np.float32(np.nan))
    return q, scale


def act8_values(q, scale):
    """The values a checkpoint stands for, float64."""
    s = np.repeat(np.asarray(scale, np.float64), BLOCK, axis=1)[:, :q.shape[1]]
    return q.astype(np.float64) * s


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob) of one row: ids by (logit descending, id ascending);
    the first top_k; the shortest prefix with top_p of their mass; those with
    p >= min_p * p_max; the first kept id, in id order, whose inclusive mass
    exceeds u times the kept mass.  (-1, -inf) for a row with nothing to draw
    from."""
    z = np.array(logits, np.float64)
    z[np.isnan(z)] = -np.inf
    m = z.max()
    if m == -np.inf:
        return -1, -np.inf
    if temperature == 0:
        return int(np.flatnonzero(z == m)[0]), 0.0
    order = np.lexsort((np.arange(z.size), -z))
    if top_k:
        order = order[:top_k]
    with np.errstate(invalid="ignore"):
        w = np.where(z[order] == m, 1.0, np.exp((z[order] - m) / temperature))
    w = np.nan_to_num(w, nan=0.0)
    if top_p < 1.0:
        c = np.cumsum(w)
        n = max(1, int((c - w < top_p * c[-1]).sum()))
        order, w = order[:n], w[:n]
    keep = (w >= min_p) & (w > 0)
    order, w = order[keep], w[keep]
    by_id = np.argsort(order)
    c = np.cumsum(w[by_id])
    i = min(int(np.searchsorted(c, u * c[-1], side="right")), len(c) - 1)
    return int(order[by_id[i]]), float(np.log(w[by_id[i]] / c[-1]))
