"""Sampling and sampled verification in 64 bits and plain Python, for the tests.

Written from the formulas of include/dflash.h; shares no code with the library."""
from __future__ import annotations

import numpy as np


def distribution(x, t):
    """Probabilities of a row of logits at a temperature, or None."""
    if not 0 <= t <= 2.0 ** 20 or np.isnan(x).any() or (x == np.inf).any() or not (x > -np.inf).any():
        return None
    if t < 2.0 ** -20:
        p = np.zeros(len(x))
        p[np.argmax(x)] = 1
        return p
    e = np.exp((x - x.max()) / t)
    return e / e.sum()


def race(r, noise):
    """(winner of r / noise, how far ahead of the next, relative)"""
    with np.errstate(divide="ignore", invalid="ignore"):
        key = np.where(r > 0, r / noise, -1.0)
    key = np.where(np.isnan(key), -1.0, key)
    i = int(np.argmax(key))
    if key[i] < 0:
        return -1, 1.0
    rest = np.delete(key, i)
    if len(rest) == 0 or rest.max() <= 0 or np.isinf(key[i]):
        return i, 1.0
    return i, float(1 - rest.max() / key[i])


def verify(parents, tokens, target, temps, draft, draft_rows, draft_temps, uniform, noise, max_path):
    """-> (path, token behind it, least margin of a comparison), or None for an entry without a result.
    target and draft: rows of logits (draft None: drafted with certainty); temps per row."""
    path, margin = [0], 1.0
    while True:
        cur = path[-1]
        p = distribution(target[cur], temps[cur])
        if p is None:
            return None
        r, found = p.copy(), None
        for c in range(cur + 1, len(parents) if len(path) < max_path else 0):
            if parents[c] != cur:
                continue
            x = tokens[c]
            if not 0 <= x < len(r):
                continue
            q = np.zeros(len(r))
            if draft is None:
                q[x] = 1
            else:
                d = draft_rows[c]
                if not 0 <= d < len(draft):
                    return None
                if 0 <= draft_temps[d] < 2.0 ** -20:
                    q[x] = 1
                else:
                    q = distribution(draft[d], draft_temps[d])
                    if q is None:
                        return None
            lhs, rhs = float(uniform[c]) * q[x], r[x]
            if max(lhs, rhs) > 0:
                margin = min(margin, abs(lhs - rhs) / max(lhs, rhs))
            if lhs < rhs:
                found = c
                break
            rest = np.maximum(r - q, 0)
            if rest.sum() > 0:
                r = rest / rest.sum()
        if found is None:
            i, m = race(r, noise)
            return (path, i, min(margin, m)) if i >= 0 else None
        path.append(found)
