"""Plain fp64 NumPy forms of the shaping of a round's logits and of the token counts it reads.

[R] "Speculative decoding", rayaq.ca ml-models -- Why the output is exactly the target's (penalties are applied to p
and q before the test). Loops over rows, positions and tokens; test infrastructure only.
"""
from __future__ import annotations

import numpy as np

from .paged_cache_oracle import tree_ok

PROMPT, MOST = 1 << 15, (1 << 15) - 1


def followed(i, parents=None):
    """The round's tokens that position i follows: a chain's before it, a tree node's line from itself to the root."""
    if parents is None:
        return list(range(i))
    line, node = [], i
    while node >= 0:
        line.append(node)
        node = int(parents[node])
    return line


def shape(logits, num=None, tokens=None, parents=None, counts=None, repetition=None, frequency=None, presence=None,
          bias_tokens=None, bias=None, mask=None):
    """(shaped, changed, size): the logits [B, N, V] after the call, where a logit was shaped, and the sum of the
    magnitudes that went into it, what its rounding errors are relative to."""
    z = np.array(logits, np.float64)
    B, N, V = z.shape
    changed, size = np.zeros(z.shape, bool), np.abs(z)
    with np.errstate(all="ignore"):
        for b in range(B):
            m = N if num is None else int(num[b])
            if not 0 <= m <= N or (parents is not None and not tree_ok(parents[b], m)):
                continue
            r = 1.0 if repetition is None else float(repetition[b])
            f = 0.0 if frequency is None else float(frequency[b])
            p = 0.0 if presence is None else float(presence[b])
            penalties = any(x is not None for x in (repetition, frequency, presence))
            for i in range(m):
                n, told = {}, set()
                if penalties:
                    if counts is not None:
                        c = np.asarray(counts[b]).astype(np.int64) & 0xffff
                        n = {int(t): int(c[t]) & MOST for t in np.nonzero(c)[0]}
                        told = {int(t) for t in np.nonzero(c & PROMPT)[0]}
                    if tokens is not None:
                        for a in followed(i, None if parents is None else parents[b]):
                            t = int(tokens[b, a])
                            if 0 <= t < V:
                                n[t] = n.get(t, 0) + 1
                for t, k in n.items():
                    x = z[b, i, t]
                    if k > 0 or t in told:
                        x = x / r if x > 0 else x * r
                    z[b, i, t] = x - f * k - (p if k > 0 else 0.0)
                    size[b, i, t] = abs(x) + abs(f) * k + abs(p)
                    changed[b, i, t] |= k > 0 or t in told
                if bias is not None:
                    for t, e in zip(bias_tokens[b], bias[b]):
                        if 0 <= t < V:
                            z[b, i, t] += float(e)
                            size[b, i, t] += abs(float(e))
                            changed[b, i, t] = True
                if mask is not None:
                    words = np.asarray(mask[b, i % mask.shape[1]]).astype(np.int64) & 0xffffffff
                    v = np.arange(V)
                    barred = (words[v // 32] >> (v % 32)) & 1 == 0
                    z[b, i, barred] = -np.inf
                    changed[b, i, barred] = True
    return z, changed, size


def count(counts, tokens, num=None, prompt=False):
    """The counts [B, V] int16 after the call (a new array)."""
    c = np.asarray(counts).astype(np.int64) & 0xffff
    B, M = tokens.shape
    for b in range(B):
        m = M if num is None else int(num[b])
        if not 0 <= m <= M:
            continue
        for t in tokens[b, :m]:
            if not 0 <= t < c.shape[1]:
                continue
            if prompt:
                c[b, t] |= PROMPT
            else:
                c[b, t] = (c[b, t] & PROMPT) | min((c[b, t] & MOST) + 1, MOST)
    return c.astype(np.uint16).view(np.int16)
