"""Accumulated attention weights and eviction (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The weight a cached position received from the accepted rows of a verification
step is the sum of its softmax probabilities over those rows and over the
query heads that read its key/value head.  Eviction keeps, per key/value head,
the most recent positions and the heaviest of the others.
"""

from __future__ import annotations

import numpy as np


def add_weights(weights, q, k, lse, prefix_len, path_len, path_nodes, scale):
    """weights [B, Hkv, S] or None; q [B, N, Hq, D], k [B, Hkv, S, D], lse
    [B, N, Hq] (base 2).  Returns (out [B, Hkv, S], lengths [B]): positions
    at or behind lengths[b] are NaN (not defined)."""
    B, N, Hq, D = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out = np.full((B, Hkv, S), np.nan)
    lens = np.zeros(B, dtype=np.int64)
    for b in range(B):
        P = min(max(int(prefix_len[b]), 0), S - N)
        n = int(path_len[b])
        nodes = (list(range(max(n, 0))) if path_nodes is None
                 else [int(x) for x in path_nodes[b][:max(n, 0)]])
        if n < 0 or n > N or any(x < 0 or x >= N for x in nodes):
            nodes = []
        lens[b] = P + len(nodes)
        for h in range(Hkv):
            acc = np.zeros(P + len(nodes))
            if weights is not None:
                acc[:P] = weights[b, h, :P]
            for t, i in enumerate(nodes):
                for g in range(h * G, h * G + G):
                    if np.isneginf(lse[b, i, g]):
                        continue
                    s = scale * (k[b, h, :P + t + 1] @ q[b, i, g])
                    acc[:P + t + 1] += np.exp(s - lse[b, i, g] * np.log(2.0))
            out[b, h, :len(acc)] = acc
    return out, lens


def kept_positions(w, length, budget, recent):
    """The kept positions of one head, ascending (w [S])."""
    length = min(max(int(length), 0), len(w))
    if length <= budget:
        return list(range(length))
    m = length - recent
    rank = sorted(range(m), key=lambda i: (-(w[i] if w[i] == w[i] else -np.inf),
                                           i))
    return sorted(rank[:budget - recent]) + list(range(m, length))
