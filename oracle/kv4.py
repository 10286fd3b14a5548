"""The 4-bit KV cache and attention over it (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A block of 16 consecutive head dims shares one scale.  With `unit` a power of
two, the block x is stored as

    scale = e4m3(max |x| / (6 unit)),  at least 2^-9, at most 448
    code  = e2m1(x / (scale unit)),    at most 6 in magnitude

each rounded to the nearest representable value, ties to the one whose last
mantissa bit is even; a code stands for unit * scale * code.  e2m1 holds
+-{0, 0.5, 1, 1.5, 2, 3, 4, 6}; e4m3 holds m 2^-9 (m < 8) and
(1 + m/8) 2^(e-7), e = 1 .. 15, up to 448.  Everything here is float64 (exact
for these sizes); rounding picks the nearest table entry.
"""

from __future__ import annotations

import numpy as np

BLOCK = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(1 + m / 8) * 2.0 ** (e - 7)
                   for e in range(1, 16) for m in range(8)][:119])


def _nearest(x, table):
    """Index of the nearest table entry to x >= 0, ties to the even index
    (in both tables the index's last bit is the mantissa's last bit)."""
    x = np.minimum(np.asarray(x, dtype=np.float64), table[-1])
    hi = np.clip(np.searchsorted(table, x), 0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = x - table[lo], table[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantise(x, unit=1.0):
    """x [..., D] -> (codes [..., D/2], scales [..., D/16]) uint8."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    bad = np.isnan(b).any(-1)
    a = np.where(np.isnan(b), 0.0, np.abs(b))
    si = np.maximum(_nearest(a.max(-1) / 6.0 / unit, E4M3), 1)
    code = _nearest(a / (E4M3[si] * unit)[..., None], E2M1)
    code = (code | (np.signbit(b) << 3)).astype(np.uint8).reshape(x.shape)
    scales = np.where(bad, 0x7F, si).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def values(codes, scales, unit=1.0):
    """The float64 values codes and scales stand for."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    table = np.concatenate([E4M3, [np.nan]])
    s = np.where(scales & 128, -1.0, 1.0) * table[scales & 127] * unit
    return v * np.repeat(s, BLOCK, -1)


def attention(q, k, v, prefix_len, mask_words, scale):
    """Tree attention with the rows' base-2 log normalisers: q [B, N, Hq, D],
    k, v [B, Hkv, S, D] float64, mask_words [B][N] ints (bit j of word i: node i
    sees drafted node j).  Returns (out, lse); a row that sees nothing gives
    zeros and -inf.  Unseen positions are not read."""
    B, N, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = np.zeros((B, N, Hq, D))
    lse = np.full((B, N, Hq), -np.inf)
    for b in range(B):
        P = int(prefix_len[b])
        for i in range(N):
            word = int(mask_words[b][i])
            keys = list(range(P)) + [P + j for j in range(N) if word >> j & 1]
            if not keys:
                continue
            for h in range(Hq):
                s = scale * (k[b, h // G, keys] @ q[b, i, h])
                m = s.max()
                w = np.exp(s - m)
                out[b, i, h] = (w / w.sum()) @ v[b, h // G, keys]
                lse[b, i, h] = (m + np.log(w.sum())) / np.log(2.0)
    return out, lse
