"""Float64 definitions of the serving operators for long contexts and drafted
tokens, one request, token or key at a time; they share no code with the
library."""
from __future__ import annotations

import math

import numpy as np

TURN = 2 * math.pi


def rotary_rates(dim, base=10000.0, scaling="none", factor=1.0, context=0.0, fast=0.0, slow=0.0):
    """(radians a position of each pair, factor of the cosines and sines)"""
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    w = [base ** (-2 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        return [x / factor for x in w], 1.0
    if scaling == "yarn":
        turns = lambda x: dim * math.log(context / (TURN * x)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(turns(fast))), min(dim - 1, math.ceil(turns(slow)))
        g = [min(1, max(0, (i - lo) / max(hi - lo, 0.001))) for i in range(dim // 2)]
        return [x * (1 - y) + x / factor * y for x, y in zip(w, g)], 0.1 * math.log(factor) + 1
    if scaling == "bands":
        g = [min(1, max(0, (context * x / TURN - slow) / (fast - slow))) for x in w]
        return [x * y + x / factor * (1 - y) for x, y in zip(w, g)], 1.0
    return w, 1.0


def rotary(x, positions, angle, layout, scale):
    """x (T, heads, D) turned; angle(position, pair) in radians."""
    x = np.array(x, dtype=np.float64)
    out = x.copy()
    n = angle.pairs
    for t, p in enumerate(positions):
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if layout == "pairs" else (i, n + i)
            c, s = scale * math.cos(angle(int(p), i)), scale * math.sin(angle(int(p), i))
            out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            out[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return out


class Angle:
    """Angles from phases (turns a position in units of 2^-64), whole turns taken off exactly."""

    def __init__(self, phases):
        self.phases, self.pairs = [int(p) % 2**64 for p in phases], len(phases)

    def __call__(self, position, i):
        return TURN * ((position * self.phases[i]) % 2**64 / 2**64)


def lse(Q, K, q_start, kv_len, table, scale, causal=True, window=0):
    """The logarithm of each row's sum of exp(scale q . k) over the keys it sees."""
    N, Hq, D = Q.shape
    n_pages, Hkv, page, _ = K.shape
    L = np.full((N, Hq), -np.inf)
    for r in range(len(kv_len)):
        a, b = int(q_start[r]), int(q_start[r + 1])
        n = min(max(0, int(kv_len[r])), table.shape[1] * page)
        k = rows_of(K, table[r], n)
        for i in range(a, b):
            lim = max(0, n - (b - i) + 1) if causal else n
            lo = max(0, lim - window) if window else 0
            if lim > lo:
                for h in range(Hq):
                    with np.errstate(all="ignore"):
                        s = k[lo:lim, h // (Hq // Hkv)] @ Q[i, h] * scale
                        m = s.max()
                        L[i, h] = m + np.log(np.exp(s - m).sum()) if m > -np.inf else m
    return L


def rows_of(K, table, n):
    """(n, heads, D) rows of a request; zeros where the table leads out of the cache."""
    n_pages, Hkv, page, D = K.shape
    out = np.zeros((n, Hkv, D))
    for j in range(n):
        pg = int(table[j // page])
        if 0 <= pg < n_pages:
            out[j] = K[pg, :, j % page]
    return out


def key_weights(Q, K, L, q_start, kv_len, held, offsets, table, weight, place, scale, causal=True):
    """Returns (weight, place)."""
    n_pages, Hkv, page, D = K.shape
    G = Q.shape[1] // Hkv
    weight, place = np.array(weight, dtype=np.float64), np.array(place)
    for r in range(len(kv_len)):
        a, b = int(q_start[r]), int(q_start[r + 1])
        n = min(max(0, int(kv_len[r])), table.shape[1] * page)
        h0 = 0 if held is None else min(max(0, int(held[r])), n)
        k = rows_of(K, table[r], n)
        w = np.zeros((n, Hkv))
        for i in range(a, b):
            lim = max(0, n - (b - i) + 1) if causal else n
            for h in range(Q.shape[1]):
                with np.errstate(all="ignore"):
                    w[:lim, h // G] += np.exp(k[:lim, h // G] @ Q[i, h] * scale - L[i, h])
        for j in range(n):
            pg = int(table[r, j // page])
            if not 0 <= pg < n_pages:
                continue
            if j < h0:
                weight[pg, :, j % page] += w[j]
            else:
                weight[pg, :, j % page] = w[j]
                place[pg, :, j % page] = j + (0 if offsets is None else int(offsets[r]))
    return weight, place


def evict(K, V, kv_len, table, weight, place, budget, recent, sinks, offsets):
    """Returns (K, V, weight, place, kept, offsets_out)."""
    K, V, weight, place = (np.array(x) for x in (K, V, weight, place))
    n_pages, Hkv, page, _ = K.shape
    kept, out = [], []
    for r in range(len(kv_len)):
        n = min(max(0, int(kv_len[r])), table.shape[1] * page)
        off = 0 if offsets is None else int(offsets[r])
        B = min(n, budget)
        kept.append(B)
        out.append(off + n - B)
        if n == B:
            continue
        at = [(int(table[r, j // page]), j % page) for j in range(n)]
        ok = [0 <= p < n_pages for p, _ in at]
        for h in range(Hkv):
            def grade(j):
                if not ok[j]:
                    return (0, 0.0)
                w, p = float(weight[at[j][0], h, at[j][1]]), int(place[at[j][0], h, at[j][1]])
                if p >= n + off - recent:
                    return (4, 0.0)
                if p < sinks:
                    return (3, 0.0)
                return (0, 0.0) if math.isnan(w) else (2, w)
            grades = [grade(j) for j in range(n)]
            stay = set(sorted(range(n), key=lambda j: (-grades[j][0], -grades[j][1], j))[:B])
            gaps, movers = [j for j in range(B) if j not in stay], [j for j in range(B, n) if j in stay]
            assert len(gaps) == len(movers)
            for d, s in zip(gaps, movers):
                if ok[d] and ok[s]:
                    for x in (K, V, weight, place):
                        x[at[d][0], h, at[d][1]] = x[at[s][0], h, at[s][1]]
    return K, V, weight, place, kept, out


def verify(target, draft, tokens, uniforms, samples, q_start, kv_len=None):
    """Returns (out with None for rows not written, accepted, kept)."""
    N, V = target.shape
    clean = lambda p: np.where(np.isnan(p), 0.0, np.clip(np.nan_to_num(p, nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0))  # noqa: E731
    out, accepted, kept = [None] * N, [], []
    for r in range(len(q_start) - 1):
        a, b = int(q_start[r]), int(q_start[r + 1])
        if b <= a:
            accepted.append(0)
            kept.append(None if kv_len is None else int(kv_len[r]))
            continue
        t = a
        while t < b - 1:
            d = int(tokens[t + 1])
            if not 0 <= d < V:
                break
            q = 1.0 if draft is None else float(clean(draft[t, d]))
            if not float(uniforms[t]) * q < float(clean(target[t, d])):
                break
            out[t] = d
            t += 1
        p = clean(target[t])
        m = p
        if t < b - 1:
            m = p.copy()
            if draft is None:
                if 0 <= int(tokens[t + 1]) < V:
                    m[int(tokens[t + 1])] = 0.0
            else:
                m = np.maximum(p - clean(draft[t]), 0.0)
            if m.sum() == 0:
                m = p
        c = np.cumsum(m)
        v = min(max(float(samples[r]), 0.0), 1 - 2.0**-24)
        out[t] = int(np.argmax(c > v * c[-1])) if c[-1] > 0 else -1
        for i in range(t + 1, b):
            out[i] = -1
        accepted.append(t - a)
        kept.append(None if kv_len is None else int(kv_len[r]) - (b - 1 - t))
    return out, accepted, kept


def trim(kv_len, kept, table, free_pages, n_free, page_size):
    """Returns (free_pages, n_free, status)."""
    free, table, status, back = [int(f) for f in free_pages], np.asarray(table), 0, []
    for r, (n, k) in enumerate(zip(kv_len, kept)):
        if n < 0 or k < 0 or k > n:
            status |= 1
            continue
        if -(-int(n) // page_size) > table.shape[1]:
            status |= 2
        back += [(r, j) for j in range(-(-int(k) // page_size), -(-int(n) // page_size))]
    if not 0 <= n_free <= len(free) or n_free + len(back) > len(free):
        status |= 4
    if status:
        return free, n_free, status
    for i, (r, j) in enumerate(back):
        free[n_free + len(back) - 1 - i] = int(table[r, j])
    return free, n_free + len(back), 0
