"""Speculative verification of drafted tokens, in long double (numpy): moe_verify_draft of k3moe_serve.h from its definition."""

from __future__ import annotations

import numpy as np

LD = np.longdouble


def probabilities(logits: np.ndarray, t: float) -> np.ndarray:
    """softmax(logits / t) of a row in long double; zeros where nothing is to be shared."""
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, LD))
    m = l.max()
    if m == -np.inf:
        return np.zeros(l.shape, LD)
    if m == np.inf:
        w = (l == np.inf).astype(LD)
    else:
        w = np.zeros(l.shape, LD)
        live = l > -np.inf
        w[live] = np.exp((l[live] - m) * (LD(0) if np.isinf(t) else 1 / LD(t)))
    return w / w.sum()


def pick(mass: np.ndarray, u: float) -> int:
    """The lowest index whose cumulative mass exceeds u times the total; -1 without mass."""
    total = np.cumsum(mass)
    if not total[-1] > 0:
        return -1
    over = np.flatnonzero((total > LD(u) * total[-1]) & (mass > 0))
    return int(over[0]) if len(over) else int(np.flatnonzero(mass > 0)[-1])


def verify_ref(logits, draft, u_accept, u_sample, probs=None, length=None, temperature=None):
    """(n_accepted [S], tokens [S, W], accept_prob [S, W-1]) of logits [S, W, V]."""
    S, W, V = logits.shape
    accepted, tokens, chance = np.zeros(S, np.int32), np.full((S, W), -1, np.int32), np.zeros((S, max(W - 1, 0)))
    for s in range(S):
        t = 1.0 if temperature is None else float(temperature[s])
        n = W - 1 if length is None else min(max(int(length[s]), 0), W - 1)
        greedy = not t > 0
        stopped = False
        for w in range(n):
            x = int(draft[s, w])
            row = np.asarray(logits[s, w], np.float64)
            if greedy:
                best = np.where(np.isnan(row), -np.inf, row)
                top = int(best.argmax()) if best.max() > -np.inf else -1
                take, chance[s, w] = x == top and top >= 0, float(x == top and top >= 0)
            else:
                p = probabilities(row, t)[x] if 0 <= x < V else LD(0)
                q = LD(1) if probs is None else LD(probs[s, w, x]) if 0 <= x < V else LD(1)
                take = LD(u_accept[s, w]) * q < p
                chance[s, w] = 1.0 if q < p else float(p / q) if q > 0 else 0.0
            if not take:
                stopped = True
            elif not stopped:
                tokens[s, w] = x
                accepted[s] += 1
        c = int(accepted[s])
        row = np.asarray(logits[s, c], np.float64)
        if greedy:
            best = np.where(np.isnan(row), -np.inf, row)
            tokens[s, c] = int(best.argmax()) if best.max() > -np.inf else -1
            continue
        mass = probabilities(row, t)
        if c < n:
            q = np.zeros(V, LD)
            if probs is not None:
                q = np.asarray(probs[s, c], LD)
            elif 0 <= int(draft[s, c]) < V:
                q[int(draft[s, c])] = 1
            left = np.maximum(mass - q, 0)
            mass = left if left.sum() > 0 else mass
        tokens[s, c] = pick(mass, float(u_sample[s]))
    return accepted, tokens, chance
