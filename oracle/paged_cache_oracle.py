"""Plain fp64 NumPy forms of the paged-cache operators: append, attention, attention weights, eviction.

[R] "Speculative decoding", rayaq.ca ml-models -- Verification attention and the cache. [B] "Inference:
distillation and speculative decoding", brunomaga.github.io -- Medusa (tree attention).

Pages are arrays [num_pages, heads, page_size, D] (weights without D), a table [B, max_pages]. Loops
over rows and tokens; test infrastructure only.
"""
from __future__ import annotations

import numpy as np


def place(table, b, j, page_size):
    return int(table[b, j // page_size]), j % page_size


def entries(pages, table, b, n):
    """Entries 0..n-1 of row b: [heads, n, ...]."""
    S = pages.shape[2]
    if n == 0:
        return pages[:0].swapaxes(0, 1).reshape(pages.shape[1], 0, *pages.shape[3:])
    return np.stack([pages[p, :, s] for p, s in (place(table, b, j, S) for j in range(n))], axis=1)


def row_ok(table, b, n, m, page_size, num_pages):
    """The row's length and pages are in range."""
    if n < 0 or m < 0 or n + m > table.shape[1] * page_size:
        return False
    return all(0 <= table[b, p] < num_pages for p in range(-(-(n + m) // page_size)))


def tree_ok(parents, m):
    return all((p == -1) if i == 0 else (0 <= p < i) for i, p in enumerate(parents[:m]))


def attended(n, m, i, parents=None):
    """The entries token i of a row attends, ascending."""
    if parents is None:
        return list(range(n + i + 1))
    line, node = [], i
    while node >= 0:
        line.append(node)
        node = int(parents[node])
    return list(range(n)) + [n + a for a in sorted(line)]


def attention(q, k, v, table, prefix, num, parents, scale):
    """(out, lse, abs): out [B, N, Hq, D], lse [B, N, Hq], and abs [B, N, Hq, D] = sum_j p_j |v_j|, what
    the errors of the probabilities are relative to. NaN for a row in error, 0 behind its tokens."""
    B, N, Hq, D = q.shape
    P, H, S, _ = k.shape
    G = Hq // H
    out, lse, mag = np.zeros(q.shape), np.zeros((B, N, Hq)), np.zeros(q.shape)
    for b in range(B):
        n, m = int(prefix[b]), int(num[b])
        if n < 0 or m < 0 or m > N or n + m > table.shape[1] * S:
            out[b], lse[b] = np.nan, np.nan
            continue
        if not row_ok(table, b, n, m, S, P) or (parents is not None and not tree_ok(parents[b], m)):
            out[b, :m], lse[b, :m] = np.nan, np.nan
            continue
        K, V = entries(k, table, b, n + m), entries(v, table, b, n + m)
        for i in range(m):
            js = attended(n, m, i, None if parents is None else parents[b])
            for h in range(Hq):
                s = scale * (K[h // G, js] @ q[b, i, h])
                mx = s.max()
                p = np.exp(s - mx)
                total = p.sum()
                lse[b, i, h] = mx + np.log(total)
                out[b, i, h] = (p / total) @ V[h // G, js]
                mag[b, i, h] = (p / total) @ np.abs(V[h // G, js])
    return out, lse, mag


def weights(q, lse, k, weight, table, prefix, num, path, scale):
    """The weight pages after a round's kept tokens have been added (a new array)."""
    B, N, Hq, D = q.shape
    P, H, S, _ = k.shape
    G = Hq // H
    weight = weight.copy()
    for b in range(B):
        n, m = int(prefix[b]), max(int(num[b]), 0) if num[b] != -1 else 0
        if n < 0 or num[b] < -1 or m > N or n + m > table.shape[1] * S:
            continue
        if path is not None and any(not 0 <= path[b, d] < N for d in range(m)):
            continue
        for j in range(n + m):
            page, slot = place(table, b, j, S)
            if not 0 <= page < P:
                continue
            for d in range(max(0, j - n), m):
                i = d if path is None else int(path[b, d])
                for h in range(Hq):
                    weight[page, h // G, slot] += np.exp(scale * (q[b, i, h] @ k[page, h // G, slot])
                                                         - lse[b, i, h])
    return weight


def kept_entries(w, budget, recent):
    """The entries of one row and head that stay, ascending: the last `recent`, and of the others the
    budget - recent with the largest weight, of equal ones the first (NaN is the largest)."""
    n = len(w)
    old = n - recent
    key = np.where(np.isnan(w[:old]), np.inf, w[:old])
    nan = np.isnan(w[:old])
    order = sorted(range(old), key=lambda j: (not nan[j], -key[j], j))
    return sorted(order[:budget - recent]) + list(range(old, n))


def evict(k, v, weight, table, length, budget, recent):
    """(k, v, weight, out_len) after the eviction (new arrays)."""
    k, v, weight = k.copy(), v.copy(), weight.copy()
    P, H, S = weight.shape
    out = []
    for b, n in enumerate(int(x) for x in length):
        if n < 0 or not row_ok(table, b, n, 0, S, P):
            out.append(-1)
            continue
        out.append(min(n, budget))
        if n <= budget:
            continue
        old = [entries(x, table, b, n) for x in (k, v, weight)]
        for h in range(H):
            for d, j in enumerate(kept_entries(old[2][h], budget, recent)):
                page, slot = place(table, b, d, S)
                for x, o in zip((k, v, weight), old):
                    x[page, h, slot] = o[h, j]
    return k, v, weight, np.array(out, np.int32)


def append(k, v, weight, k_new, v_new, table, prefix, num, path):
    """(k, v, weight, out_len) after the round's entries were written (new arrays)."""
    k, v = k.copy(), v.copy()
    weight = None if weight is None else weight.copy()
    P, _, S, _ = k.shape
    N = k_new.shape[1]
    out = []
    for b in range(len(prefix)):
        n, m = int(prefix[b]), int(num[b])
        m = 0 if m == -1 else m
        ok = n >= 0 and 0 <= m <= N and n + m <= table.shape[1] * S
        ok = ok and all(0 <= place(table, b, n + d, S)[0] < P for d in range(m))
        ok = ok and (path is None or all(0 <= path[b, d] < N for d in range(m)))
        out.append(n + m if ok else -1)
        for d in range(m if ok else 0):
            page, slot = place(table, b, n + d, S)
            i = d if path is None else int(path[b, d])
            k[page, :, slot], v[page, :, slot] = k_new[b, i], v_new[b, i]
            if weight is not None:
                weight[page, :, slot] = 0
    return k, v, weight, np.array(out, np.int32)
