"""Oracle of what surrounds a layer's products (TEST INFRASTRUCTURE ONLY): the
root-mean-square norm with the residual's addition, and the routing of tokens
to experts, in float64."""
from __future__ import annotations

import numpy as np


def rms_norm(x, weight, eps, residual=None, weight_offset=0.0):
    """x [..., K] -> (y, h): h = x + residual, y = h / sqrt(mean(h^2) + eps) * (weight + offset)."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    r = 1.0 / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)
    return h * r * (np.asarray(weight, np.float64) + weight_offset), h


def scores(logits, score):
    x = np.asarray(logits, np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    top = x.max(axis=1, keepdims=True)
    e = np.exp(x - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(axis=1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def route(logits, topk, score="softmax", bias=None, num_groups=1, topk_groups=1, group_score="max", renormalize=True,
          scale=1.0):
    """-> (ids int64 [T, topk], weights float64 [T, topk]), one token and one choice at a time."""
    x = np.asarray(logits, np.float64)
    t, e = x.shape
    s = scores(x, score)
    key = x.copy() if bias is None else np.where(x == -np.inf, -np.inf, s + np.asarray(bias, np.float64))
    ids, w = np.full((t, topk), -1, np.int64), np.zeros((t, topk))
    n = e // num_groups
    for i in range(t):
        left = {j: key[i, j] for j in range(e) if key[i, j] > -np.inf}
        if num_groups > 1:
            order = []
            for g in range(num_groups):
                mine = sorted((s[i, j] if bias is None and group_score == "top2" else left[j]
                               for j in range(g * n, (g + 1) * n) if j in left), reverse=True)
                of = -np.inf if not mine else sum(mine[:2]) if group_score == "top2" else mine[0]
                order.append((-of, g))
            kept = {g for _, g in sorted(order)[:topk_groups]}
            left = {j: v for j, v in left.items() if j // n in kept}
        best = sorted(left, key=lambda j: (-left[j], j))[:topk]
        ids[i, :len(best)] = best
        w[i, :len(best)] = s[i, best]
        if renormalize and w[i].sum() > 0:
            w[i] /= w[i].sum()
    return ids, w * scale
