"""Float64 NumPy definitions of the serving operators, one request, token or
key at a time; they share no code with the library."""
from __future__ import annotations

import numpy as np


def paged_plan(cached, fresh, table, free_pages, n_free, page_size, n_tokens, capacity=None):
    """Returns (q_start, kv_len, slots, token_req, positions, table, n_free, status)."""
    cached, fresh = [int(c) for c in cached], [int(f) for f in fresh]
    capacity = len(free_pages) if capacity is None else capacity
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    status = 0
    want = 0
    for c, f in zip(cached, fresh):
        if c < 0 or f < 0 or c + f > 2**31 - 1:
            status |= 1
            continue
        if -(-(c + f) // page_size) > width:
            status |= 2
        want += -(-(c + f) // page_size) - -(-c // page_size)
    if not 0 <= n_free <= capacity or want > n_free:
        status |= 4
    if sum(f for c, f in zip(cached, fresh) if c >= 0 and f >= 0 and c + f < 2**31) > n_tokens:
        status |= 8
    slots, reqs, places = ([-1] * n_tokens for _ in range(3))
    if status:
        return ([0] * (len(cached) + 1), [max(0, c) for c in cached], slots, reqs, places, table, n_free, status)
    starts, t = [0], 0
    for r, (c, f) in enumerate(zip(cached, fresh)):
        for p in range(c, c + f):
            if p % page_size == 0:
                n_free -= 1
                table[r, p // page_size] = free_pages[n_free]
            page = table[r, p // page_size]
            slots[t] = -1 if page < 0 else int(page) * page_size + p % page_size
            reqs[t], places[t] = r, p
            t += 1
        starts.append(t)
    return (starts, [c + f for c, f in zip(cached, fresh)], slots, reqs, places, table, n_free, 0)


def keys_of(q_len, kv_len, i, causal, window):
    """The range of keys that token i of a chunk sees."""
    lim = max(0, kv_len - q_len + i + 1) if causal else kv_len
    return (max(0, lim - window) if window else 0), lim


def attention(Q, K, V, q_start, kv_len, table, scale, causal=True, window=0):
    """Q (N, Hq, D), K and V (pages, Hkv, page, D) in float64.  Returns (O, A, rows):
    O as the operator defines it, A = sum_j p_j |v_j| (the scale of its rounding
    errors) and the mask of rows that belong to a request."""
    N, Hq, D = Q.shape
    n_pages, Hkv, page, _ = K.shape
    G = Hq // Hkv
    O, A = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    rows = np.zeros(N, dtype=bool)
    for r in range(len(kv_len)):
        a, b = int(q_start[r]), int(q_start[r + 1])
        n = min(max(0, int(kv_len[r])), table.shape[1] * page)
        rows[a:b] = True
        if b <= a:
            continue
        ks, vs = np.zeros((n, Hkv, D)), np.zeros((n, Hkv, D))
        for j in range(n):
            pg = int(table[r, j // page])
            if 0 <= pg < n_pages:
                ks[j], vs[j] = K[pg, :, j % page], V[pg, :, j % page]
        for i in range(b - a):
            lo, lim = keys_of(b - a, n, i, causal, window)
            if lim <= lo:
                continue
            for h in range(Hq):
                k, v = ks[lo:lim, h // G], vs[lo:lim, h // G]
                with np.errstate(all="ignore"):
                    s = (k @ Q[a + i, h]) * scale
                    p = np.exp(s - s.max())
                    p = p / p.sum()
                    O[a + i, h] = (p[:, None] * v).sum(0)
                    A[a + i, h] = (p[:, None] * np.abs(v)).sum(0)
    return O, A, rows


def norm(v, kind, weight=None, bias=None, eps=1e-5):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdims=True)
    v = v / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    if weight is not None:
        v = v * weight
    return v if bias is None else v + bias


def norm_residual(h, y, alpha, post, gate, gate_index, pre):
    """post, pre: (kind, weight, bias, eps) or None.  Returns (h', x)."""
    out = alpha * h
    if y is not None:
        y = norm(y, *post) if post else y
        if gate is not None:
            index = np.zeros(len(h), dtype=int) if gate_index is None else np.asarray(gate_index)
            g = np.zeros_like(h)
            for t, i in enumerate(index):
                if 0 <= i < len(gate):
                    g[t] = gate[i]
            y = g * y
        out = out + y
    return out, (norm(out, *pre) if pre else out)
