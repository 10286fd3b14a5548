"""Log probabilities of given tokens, entropy, alternatives, gradient (oracle
side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

p = softmax(z / T) per row, in float64: ln p of the given tokens, H = -sum p ln
p, the most probable tokens (equal logits by lower index), and the gradient of
sum_j g_j ln p(t_j) + g_H H with respect to the logits.
"""

from __future__ import annotations

import numpy as np


def log_softmax(z, T):
    """ln p of every token, and the natural log normaliser, row by row.  (The
    maximum is taken off first: beside logits of 1e20 it would swallow ln S.)"""
    z = np.asarray(z, dtype=np.float64) / T
    m = z.max(-1, keepdims=True)
    ln = np.log(np.exp(z - m).sum(-1, keepdims=True))
    return z - m - ln, (m + ln)[..., 0]


def token_logprobs(z, tokens, T=1.0, top=0):
    """z [M, V], tokens [M, n].  Returns (logprob [M, n], base-2 lse [M],
    entropy [M], ids [M, top], their logprobs [M, top])."""
    lp, lse = log_softmax(z, T)
    p = np.exp(lp)
    H = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(-1)
    M, V = lp.shape
    out = np.zeros(tokens.shape)
    for i in range(M):
        for j, x in enumerate(tokens[i]):
            if 0 <= x < V:
                out[i, j] = lp[i, x]
    ids = np.argsort(-np.asarray(z, dtype=np.float64), axis=-1,
                     kind="stable")[:, :top]
    return (out, lse / np.log(2.0), H, ids, np.take_along_axis(lp, ids, -1))


def grad(z, tokens, g_logprob, g_entropy=None, T=1.0):
    """dL/dz of L = sum g_logprob ln p(tokens) + g_entropy H, [M, V]."""
    lp, _ = log_softmax(z, T)
    p = np.exp(lp)
    M, V = lp.shape
    d = np.zeros((M, V))
    for i in range(M):
        for j, x in enumerate(tokens[i]):
            if 0 <= x < V:
                d[i] -= g_logprob[i, j] * p[i]
                d[i, x] += g_logprob[i, j]
        if g_entropy is not None:
            l = np.where(p[i] > 0, lp[i], 0.0)
            H = -(p[i] * l).sum()
            d[i] -= g_entropy[i] * p[i] * (l + H)
    return d / T
