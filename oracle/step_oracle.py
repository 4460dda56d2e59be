"""Plain CPU definition (NumPy, fp64) of what a decode step does with rows between its
products: what the kernels behind include/qgstep.h have to give.

Token by token and element by element where that says it most plainly; it shares no
code with the HIP path.
"""
from __future__ import annotations

import math

import numpy as np


def rms_norm(h, weight=None, eps: float = 1e-6) -> np.ndarray:
    """Rows [rows][n], already summed with the residual and rounded as they are stored."""
    h = np.asarray(h, dtype=np.float64)
    with np.errstate(all="ignore"):
        y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return y if weight is None else y * np.asarray(weight, dtype=np.float64)


def group_scales(y, top: float, group: int = 0) -> np.ndarray:
    """[rows][groups]: the largest magnitude of each over `top`."""
    n = y.shape[1]
    g = group or n
    return np.stack([np.abs(y[:, a:a + g]).max(-1) / top for a in range(0, n, g)], 1)


def rotate(x, positions, freqs, size: float = 1.0, pairs: bool = False) -> np.ndarray:
    """x [rows][heads][head_dim]; pair j turned by positions * freqs[j] radians."""
    out = np.array(x, dtype=np.float64)
    d = 2 * len(freqs)
    for i, p in enumerate(positions):
        for j, f in enumerate(freqs):
            a, b = (2 * j, 2 * j + 1) if pairs else (j, j + d // 2)
            c, s = size * math.cos(int(p) * f), size * math.sin(int(p) * f)
            u, v = out[i, :, a].copy(), out[i, :, b].copy()
            out[i, :, a], out[i, :, b] = u * c - v * s, u * s + v * c
    return out


def kept_tokens(logits, temperature: float, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """The kept tokens of one row in their order (falling logit, rising index) and their weights."""
    l = np.array(logits, dtype=np.float64)
    l[np.isnan(l)] = -np.inf
    order = sorted((i for i in range(l.size) if l[i] > -np.inf), key=lambda i: (-l[i], i))
    if not order:
        return [], np.zeros(0)
    if not temperature > 0:
        return order[:1], np.ones(1)
    top = l[order[0]]
    w = np.array([1.0 if l[i] == top else math.exp((l[i] - top) / temperature) for i in order])
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    if top_p < 1:
        total, run, n = w.sum(), 0.0, 0
        while n < len(order) and (n == 0 or run < top_p * total):
            run += w[n]
            n += 1
        order, w = order[:n], w[:n]
    keep = [j for j in range(len(order)) if w[j] >= min(min_p, 1.0) or j == 0]
    return [order[j] for j in keep], w[keep]


def sample(logits, u: float, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """(token, probability) of one row; (-1, 0) where there is no token."""
    order, w = kept_tokens(logits, temperature, top_k, top_p, min_p)
    if not order:
        return -1, 0.0
    by = np.argsort(order, kind="stable")
    run = np.cumsum(w[by])
    j = min(int(np.searchsorted(run, min(max(u, 0.0), 1.0) * run[-1], side="right")), len(by) - 1)
    return order[by[j]], float(w[by[j]] / run[-1])
