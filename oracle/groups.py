"""Grouped top-k routing, in fp64 (numpy): moe_route_groups of k3moe_serve.h from its definition."""

from __future__ import annotations

import numpy as np

from oracle.route import sigmoid64


def gates(z: np.ndarray, score: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if score == "sigmoid":
        return sigmoid64(z)
    m = np.where(np.isnan(z), -np.inf, z).max(-1, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(z == m, 1.0, np.where(m == np.inf, 0.0, np.exp(z - m)))
    w = np.where(z == -np.inf, 0.0, np.where(np.isnan(z), np.nan, w))
    total = np.nansum(w, -1, keepdims=True)
    return w / np.where(total > 0, total, 1.0)


def route_groups_ref(z, bias, k, groups, keep, group_top=2, score="sigmoid", normalize=True, route_scale=1.0):
    """ids int32 [T, k], weights fp32 [T, k] of logits z [T, E]."""
    z = np.asarray(z)
    T, E = z.shape
    n = E // groups
    g = gates(z, score)
    s = g if bias is None else g + np.asarray(bias, dtype=np.float64)[None]
    s = np.where(np.isnan(s), -np.inf, s)
    best = np.sort(s.reshape(T, groups, n), -1)[..., ::-1][..., :group_top]
    with np.errstate(invalid="ignore"):
        gs = best.sum(-1)
    gs = np.where(np.isnan(gs), -np.inf, gs)
    ids = np.zeros((T, k), np.int32)
    for t in range(T):
        kept = sorted(range(groups), key=lambda i: (-gs[t, i], i))[:keep]
        among = [e for i in kept for e in range(i * n, (i + 1) * n)]
        ids[t] = sorted(among, key=lambda e: (-s[t, e], e))[:k]
    w = np.take_along_axis(g, ids.astype(np.int64), 1)
    if normalize:
        total = w.sum(1, keepdims=True)
        w = np.where(total == 0, 0.0, w / np.where(total == 0, 1.0, total))
    return ids, (w * float(np.float32(route_scale))).astype(np.float32)
