"""fp64 CPU oracle of the paged key-value cache (test infrastructure, like
gsi_oracle: the library never calls it and shares no code with it): rotary
positions, appending, attention of one token, eviction.

Every function is a loop over the definition in gsi.h.  A pool is a dict of
numpy arrays K, V [pages][heads][page][d] and mass, age [pages][heads][page]
(or None)."""
from __future__ import annotations

import math

import numpy as np


def rotary(x, positions, freq, layout: str, start: int = 0, amplitude: float = 1.0) -> np.ndarray:
    """x [T][heads][d] with its pairs turned; layout "pairs" or "halves"."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = len(freq)
    for t in range(x.shape[0]):
        for i in range(half):
            a = math.fmod(float(int(positions[t])) * float(freq[i]), 2 * math.pi)
            c, s = amplitude * math.cos(a), amplitude * math.sin(a)
            e0, e1 = (start + 2 * i, start + 2 * i + 1) if layout == "pairs" else (start + i, start + half + i)
            y[t, :, e0] = x[t, :, e0] * c - x[t, :, e1] * s
            y[t, :, e1] = x[t, :, e1] * c + x[t, :, e0] * s
    return y


def _place(pool, row, i):
    """(page, slot of the page) of slot i of the sequence with the page numbers `row`, or None."""
    pages, page = pool["K"].shape[0], pool["K"].shape[2]
    if not 0 <= i < len(row) * page:
        return None
    p = int(row[i // page])
    return (p, i % page) if 0 <= p < pages else None


def append(pool, table, seq, slots, k, v, positions=None):
    """k (as it is stored) and v [T][heads][d] into the pool, in place."""
    for t in range(len(slots)):
        s = t if seq is None else int(seq[t])
        at = _place(pool, table[s], int(slots[t])) if 0 <= s < len(table) else None
        if at is None:
            continue
        p, o = at
        pool["K"][p, :, o], pool["V"][p, :, o] = k[t], v[t]
        if pool["mass"] is not None:
            pool["mass"][p, :, o] = 0.0
        if pool["age"] is not None:
            age = int(slots[t]) if positions is None else int(positions[t])
            pool["age"][p, :, o] = min(max(age, -2**31), 2**31 - 1)


def attend(pool, table, lengths, q, scale: float, window: int = 0):
    """(out, lse, weights added to mass, sum of weight |v|, largest scale sum |q k|
    of a head) for q [S][heads][d]."""
    S, H, d = q.shape
    heads, page = pool["K"].shape[1:3]
    out, lse, size = np.zeros((S, H, d)), np.full((S, H), -np.inf), np.zeros((S, H, d))
    big = np.zeros((S, H))
    mass = np.zeros(pool["K"].shape[:3])
    for s in range(S):
        n = min(max(int(lengths[s]), 0), len(table[s]) * page)
        first = max(0, n - window) if window else 0
        at = [a for a in (_place(pool, table[s], i) for i in range(first, n)) if a is not None]
        if not at:
            continue
        p, o = np.array([a[0] for a in at]), np.array([a[1] for a in at])
        for h in range(H):
            kh = h // (H // heads)
            k = np.asarray(pool["K"][p, kh, o], dtype=np.float64)
            v = np.asarray(pool["V"][p, kh, o], dtype=np.float64)
            score = scale * (k @ q[s, h])
            top = score.max()
            if top == -np.inf:
                continue
            e = np.exp(score - top)
            w = e / e.sum()
            lse[s, h] = top + math.log(e.sum())
            out[s, h], size[s, h] = w @ v, w @ np.abs(v)
            big[s, h] = abs(scale) * (np.abs(k) @ np.abs(q[s, h])).max()
            np.add.at(mass, (p, kh, o), w)
    return out, lse, mass, size, big


def evict(pool, table, lengths, budget: int, recent: int):
    """(lengths_out [S], from [S][heads][budget]); the pool is left as it is."""
    S, heads, page = len(table), pool["K"].shape[1], pool["K"].shape[2]
    out, source = np.zeros(S, np.int32), np.full((S, heads, budget), -1, np.int32)
    for s in range(S):
        n = min(max(int(lengths[s]), 0), len(table[s]) * page)
        out[s] = min(n, budget)
        for h in range(heads):
            if n <= budget:
                source[s, h, :n] = range(n)
                continue
            at = [_place(pool, table[s], i) for i in range(n)]

            def age(i):
                if pool["age"] is None:
                    return i
                return -2**31 if at[i] is None else int(pool["age"][at[i][0], h, at[i][1]])

            def mass(i):
                m = None if at[i] is None else float(pool["mass"][at[i][0], h, at[i][1]])
                return (0, 0.0) if m is None or math.isnan(m) else (1, m)

            newest = sorted(range(n), key=lambda i: (-age(i), i))
            rest = sorted(newest[recent:], key=lambda i: (-mass(i)[0], -mass(i)[1], i))
            keep = set(newest[:recent]) | set(rest[:budget - recent])
            behind = iter(sorted(i for i in keep if i >= budget))
            for j in range(budget):
                source[s, h, j] = j if j in keep else next(behind)
    return out, source


def move(pool, table, source, to=None):
    """Every entry to the slot that `source` gives it, in place."""
    old = {k: None if v is None else v.copy() for k, v in pool.items()}
    S, heads, budget = source.shape
    for s in range(S):
        for h in range(heads):
            for j in range(budget):
                i = int(source[s, h, j])
                if i < 0 or (to is None and i == j):
                    continue
                a, b = _place(pool, table[s], i), _place(pool, (table if to is None else to)[s], j)
                if a is None or b is None:
                    continue
                for name in pool:
                    if pool[name] is not None:
                        pool[name][b[0], h, b[1]] = old[name][a[0], h, a[1]]
