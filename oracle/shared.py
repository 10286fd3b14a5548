"""Tree attention of sequences that share a prefix (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A sequence's keys are its prefix's shared positions, its own positions and the
drafted nodes; node i sees the first two and the nodes of its mask row.  float64.
"""

from __future__ import annotations

import numpy as np

from .prompt import attend


def tree_attention_shared(q, kp, vp, shared_len, group_start, k, v, prefix_len,
                          bits, scale):
    """q [B, N, Hq, D]; kp, vp [groups, Hkv, Sp, D]; k, v [B, Hkv, S, D]; bits
    [B, N] uint64.  Returns out, lse and the two magnitudes of `attend`
    ([B, N, Hq, D], [B, N, Hq], [B, N, Hq, D], [B, N, Hq]); sequences outside
    every group stay NaN."""
    B, N, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mag = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, sm = np.full((B, N, Hq), np.nan), np.full((B, N, Hq), np.nan)
    for g in range(len(shared_len)):
        n = min(max(int(shared_len[g]), 0), kp.shape[2])
        for b in range(max(int(group_start[g]), 0),
                       min(int(group_start[g + 1]), B)):
            P = min(max(int(prefix_len[b]), 0), k.shape[2] - N)
            sees = np.ones((N, n + P + N), dtype=bool)
            for i in range(N):
                for j in range(N):
                    sees[i, n + P + j] = (int(bits[b, i]) >> j) & 1
            for h in range(Hq):
                kk = np.concatenate([kp[g, h // G, :n], k[b, h // G, :P + N]])
                vv = np.concatenate([vp[g, h // G, :n], v[b, h // G, :P + N]])
                out[b, :, h], lse[b, :, h], mag[b, :, h], sm[b, :, h] = attend(
                    q[b, :, h], kk, vv, scale, sees)
    return out, lse, mag, sm
