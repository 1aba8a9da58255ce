"""The target model's side in 64 bits and plain Python, for the tests: rotary
positions, attention of a tree over pages, trees, and the cache's pages.

Written from the formulas of include/dflash.h; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np


def rope_freqs(rd, theta=1e6, scaling="none", factor=1.0, orig=0, beta_fast=32.0, beta_slow=1.0, mscale=0.0):
    """(angle per position of every pair, magnitude factor)"""
    if scaling == "ntk":
        theta = theta * factor ** (rd / (rd - 2))
    f = [theta ** (-2 * j / rd) for j in range(rd // 2)]
    m = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "yarn":
        def dim(b):
            return rd * math.log(orig / (2 * math.pi * b)) / (2 * math.log(theta))
        lo, hi = max(math.floor(dim(beta_fast)), 0), min(math.ceil(dim(beta_slow)), rd - 1)
        w = [min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for j in range(rd // 2)]
        f = [x * (a / factor + 1 - a) for x, a in zip(f, w)]
        if factor > 1:
            m = 0.1 * math.log(factor) + 1
    return np.array(f, dtype=np.float64), mscale or m


def rope(x, pos, layout, rd, freqs, m, backward=False):
    """x [T][heads][hd] float64 -> rotated, float64; also the bound's |a| + |b| per element."""
    y, size = x.copy(), np.abs(x)
    if rd == 0:
        return y, size
    t = pos.astype(np.float64)[:, None] * freqs
    c, s = np.cos(t)[:, None] * m, np.sin(t)[:, None] * m
    if backward:
        s = -s
    a, b = (slice(0, rd // 2), slice(rd // 2, rd)) if layout == "half" else (slice(0, rd, 2), slice(1, rd, 2))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * m
    return y, size


def tree_sets(parents):
    """Ancestor-or-self sets of one tree as a boolean matrix."""
    n = len(parents)
    m = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def words_of(m, words):
    """Boolean [n][k] -> int32 [n][words]"""
    out = np.zeros((m.shape[0], words), dtype=np.uint32)
    for i, j in zip(*np.nonzero(m)):
        out[i, j // 32] |= np.uint32(1 << (j % 32))
    return out.view(np.int32)


def attend(q, k, v, sees, scale):
    """q [n][hq][hd], k and v [slots][hkv][hd], sees [n][slots], all 64 bits.
    -> out, lse, sum of w |v| and max of scale |q| |k| over attended slots (the error bound's terms)"""
    n, hq, hd = q.shape
    g = hq // k.shape[1]
    out, lse = np.zeros((n, hq, hd)), np.full((n, hq), -np.inf)
    size, big = np.zeros((n, hq, hd)), np.zeros((n, hq))
    for h in range(hq):
        kk, vv = k[:, h // g], v[:, h // g]
        for i in range(n):
            on = np.nonzero(sees[i])[0]
            if len(on) == 0:
                continue
            s = kk[on] @ q[i, h] * scale
            top = s.max()
            e = np.exp(s - top)
            w = e / e.sum()
            out[i, h], lse[i, h] = w @ vv[on], top + np.log(e.sum())
            size[i, h] = w @ np.abs(vv[on])
            big[i, h] = (np.abs(kk[on]) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, size, big


def attend_bounds(out, size, big, slots, hd, dtype):
    """Largest error of (out, lse) that the number formats allow.

    Scores: hd products summed in fp32, (hd + 2) 2^-24 of scale |q| |k|; f32
    operands may be multiplied in pieces that keep 2^-20 of each product.  A
    score off by d moves a weight by a factor e^d and the sum by as much.  The
    exponential and its argument (a score times log2 e, of magnitude up to `big`)
    add 2^-22 + big 2^-23.  Weights may be rounded to the storage type for the
    product with the values (bf16: half a step, 2^-8), products and the sum of
    up to `slots` of them are fp32.  The result is rounded once."""
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    piece = 0.0 if dtype == "bf16" else 2.0 ** -20
    d = big * ((hd + 2) * 2.0 ** -24 + piece + 2.0 ** -23) + 2.0 ** -22
    w = (2.0 ** -8 if dtype == "bf16" else piece) + (slots + 8) * 2.0 ** -24
    tol = half * np.abs(out) * 1.01 + size * (2.02 * d[..., None] + w) + 1e-30
    return tol, d * 1.01 + (slots + 8) * 2.0 ** -24 + 2.0 ** -23 * (1 + big)


def accept(parents, tokens, targets, max_path):
    """(path, target's token after it) of one tree"""
    path = [0]
    while len(path) < max_path:
        cur = path[-1]
        nxt = [i for i in range(cur + 1, len(parents)) if parents[i] == cur and tokens[i] == targets[cur]]
        if not nxt:
            break
        path.append(nxt[0])
    return path, targets[path[-1]]


class Pages:
    """Table, lengths and reference counts in plain Python, one entry after another."""

    def __init__(self, n_pages, max_seq, max_pages, ps):
        self.ps, self.max_pages = ps, max_pages
        self.table = [[-1] * max_pages for _ in range(max_seq)]
        self.length = [0] * max_seq
        self.refs = [0] * n_pages
        self.copies = []   # (from, to, slots) of the last reserve

    def reserve(self, seqs, count):
        table, refs = [list(t) for t in self.table], list(self.refs)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        copies, seen = [], set()
        for q, c in zip(seqs, count):
            if q in seen or not 0 <= q < len(table) or c <= 0:
                seen.add(q)
                continue
            seen.add(q)
            n = self.length[q]
            for idx in range(n // self.ps, (n + c - 1) // self.ps + 1):
                if idx >= self.max_pages:
                    return False
                had, fill = table[q][idx], n - idx * self.ps
                if had >= 0 and not (fill > 0 and refs[had] > 1):
                    continue
                if not free:
                    return False
                p = free.pop(0)
                refs[p] = 1
                if had >= 0:
                    refs[had] -= 1
                    copies.append((had, p, fill))
                table[q][idx] = p
        self.table, self.refs, self.copies = table, refs, copies
        return True

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            for i in range(-(-self.length[a] // self.ps)):
                p = self.table[b][i] = self.table[a][i]
                self.refs[p] += 1
            self.length[b] = self.length[a]

    def trim(self, seqs, new_len):
        for q, n in zip(seqs, new_len):
            self.length[q] = min(self.length[q], n)
            for i in range(-(-n // self.ps), self.max_pages):
                if self.table[q][i] >= 0:
                    self.refs[self.table[q][i]] -= 1
                    self.table[q][i] = -1
