"""Verification of drafted tokens, plain -- TEST INFRASTRUCTURE ONLY.

Written from the definition (include/moe_gb300.h) in numpy: loops over sequences
and tokens, fp64 probabilities.  Shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def target(logits, temperature: float) -> np.ndarray:
    """p of one row, fp64.  Logits that are no numbers have no probability; infinity
    counts as the largest finite fp32 number."""
    z = np.asarray(logits, np.float64).copy()
    z[np.isnan(z)] = -np.inf
    z = np.minimum(z, np.finfo(np.float32).max)
    if not temperature > 0:
        p = np.zeros(len(z))
        p[np.argmax(z)] = 1.0  # the first of equal ones
        return p
    e = np.exp((z - z.max()) / temperature)
    return e / e.sum()


def draw(weights, u: float) -> int:
    """The first index whose running sum passes u times the whole."""
    run = np.cumsum(weights)
    past = np.flatnonzero((run > u * run[-1]) & (weights > 0))
    return int(past[0]) if len(past) else int(np.flatnonzero(weights > 0)[-1])


def verify(logits, tokens, q_offsets, u, u_next, draft_probs=None, temperature=None):
    """(accepted, token, refused, near, gap): lists over the sequences.  near: the least
    distance of u q(x) from p(x), relative to p(x); gap: the least distance of a running
    sum of the next token's probabilities (not brought to a whole of 1) from the number
    that it was compared with."""
    V, result = logits.shape[1], []
    for b in range(len(q_offsets) - 1):
        t0, t1 = int(q_offsets[b]), int(q_offsets[b + 1])
        if t1 == t0:
            result.append((0, -1, 0, np.inf, np.inf))
            continue
        temp = 1.0 if temperature is None else float(temperature[b])
        n, i, near, rest = t1 - t0 - 1, 0, np.inf, None
        while True:
            p = target(logits[t0 + i], temp)
            if i == n:
                rest = p
                break
            x = int(tokens[t0 + i + 1])
            ok = 0 <= x < V
            q = draft_probs[t0 + i].astype(np.float64) if draft_probs is not None else np.zeros(V)
            if draft_probs is None and ok:
                q[x] = 1.0
            uq, px = float(u[t0 + i + 1]) * (q[x] if ok else 0.0), p[x] if ok else 0.0
            if ok and px > 0:
                near = min(near, abs(uq / px - 1))
            if ok and uq < px:
                i += 1
                continue
            rest = np.maximum(p - q, 0)
            if rest.sum() == 0:
                rest = p
            break
        run = np.cumsum(rest)
        gap = np.abs(run - float(u_next[b]) * run[-1]).min() if temp > 0 else np.inf
        result.append((i, draw(rest, float(u_next[b])), n - i, near, gap))
    return [list(x) for x in zip(*result)] if result else [[], [], [], [], []]
