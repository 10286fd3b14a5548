"""Causal attention of packed prompts (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Token i of a prompt attends to the prompt's tokens 0 .. i; query head h reads
key/value head h // (Hq / Hkv).  float64.
"""

from __future__ import annotations

import numpy as np


def attend(q, k, v, scale, sees):
    """q [R, D], k, v [L, D], sees [R, L] -> outputs [R, D], base-2 normalisers
    [R], sum of weighted magnitudes of v [R, D], largest scale sum |q_d k_d| of
    a visible key [R].  A row that sees nothing gives zeros and -inf."""
    s = np.where(sees, scale * (q @ k.T), -np.inf)
    m = s.max(-1, initial=-np.inf, keepdims=True)
    w = np.exp(s - np.where(np.isneginf(m), 0.0, m))
    l = w.sum(-1, keepdims=True)
    p = w / np.where(l > 0, l, 1.0)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0] / np.log(2.0)
    mag = np.where(sees, scale * (np.abs(q) @ np.abs(k).T), 0.0)
    return p @ v, lse, p @ np.abs(v), mag.max(-1, initial=0.0)


def prompt_attention(q, k, v, starts, scale):
    """q [T, Hq, D]; k, v [T, Hkv, D]; starts [B+1].  Returns out, lse and the
    two magnitudes of `attend` ([T, Hq, D], [T, Hq], [T, Hq, D], [T, Hq]);
    tokens outside every prompt stay NaN."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mag = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    lse, sm = np.full((T, Hq), np.nan), np.full((T, Hq), np.nan)
    for a, z in zip(starts, starts[1:]):
        if z <= a:
            continue
        sees = np.tril(np.ones((z - a, z - a), dtype=bool))
        for h in range(Hq):
            out[a:z, h], lse[a:z, h], mag[a:z, h], sm[a:z, h] = attend(
                q[a:z, h], k[a:z, h // G], v[a:z, h // G], scale, sees)
    return out, lse, mag, sm
