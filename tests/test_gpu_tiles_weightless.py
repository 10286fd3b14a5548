"""Infinite values of keys that a row sees with a weight of 0 -- a score of -inf,
or so far below the row's largest that the exponential is 0 -- arrive as 0 times
infinity, NaN, wherever a key block or a cut between pieces lies.  Scores are made
of ones and constants, so a weight is either 1 in n or e^-500 and less.
"""

import pytest
import torch

from tests._parity import lib_ready
from tests.test_gpu_prompt import api, i32
from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def sink(k, score):
    """Makes a key's score against ones `score` or -inf."""
    if score == -INF:
        k[..., 3] = -INF
    else:
        k[...] = score / k.shape[-1]


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("score", [-512.0, -INF])
def test_prompts(score, D):
    T = 900
    q = torch.ones(T, 8, D, device="cuda").bfloat16()
    v = torch.randn(T, 2, D, device="cuda").bfloat16()
    start = i32([0, T])
    for pos in (0, 1, 63, 64, 127, 128, 200, 640, 899):
        k = torch.zeros(T, 2, D, device="cuda").bfloat16()
        sink(k[pos, 1], score)
        base, lse0 = api().spec_prompt_attention(q, k, v, start, scale=1.0,
                                                 lse=True)
        v2 = v.clone()
        v2[pos, 1, 5], v2[pos, 1, D - 1] = INF, -INF
        out, lse = api().spec_prompt_attention(q, k, v2, start, scale=1.0,
                                               lse=True)
        want = base.clone()
        want[pos:, 4:, [5, D - 1]] = float("nan")
        if pos == 0 and score != -INF:    # the only key that token 0 sees
            want[0, 4:, 5], want[0, 4:, D - 1] = INF, -INF
        assert torch.equal(lse, lse0)
        assert torch.equal(torch.nan_to_num(out, 77., 88., 99.),
                           torch.nan_to_num(want, 77., 88., 99.)), pos


def uniform(slen, pre, N, D, seed):
    c = Case([slen], [0, len(pre)], pre, N, 8, 2, D, seed=seed)
    c.q[:] = 1
    for t in (c.kp, c.k):
        t[~torch.isnan(t)] = 0
    c.scale = 1.0
    return c


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("score", [-512.0, -INF])
@pytest.mark.parametrize("slen", [300, 7000])
def test_shared_prefixes(slen, score, D):
    pre, N = [50, 0, 130, 300], 2
    c = uniform(slen, pre, N, D, 1)
    norm = lambda t: torch.nan_to_num(t, 77., 88., 99.)
    at = [(c.kp, c.vp, 0, p) for p in (0, 127, 128, slen - 1)]
    at += [(c.k, c.v, b, p) for b, p in ((0, 0), (2, 127), (2, 128), (3, 299))]
    for k, v, b, pos in at:
        kept, had = k[b, 1, pos].clone(), v[b, 1, pos, 5].clone()
        sink(k[b, 1, pos], score)
        base, lse0 = c.run()
        v[b, 1, pos, 5] = INF
        out, lse = c.run()
        k[b, 1, pos], v[b, 1, pos, 5] = kept, had
        want = base.clone()
        (want if k is c.kp else want[b:b + 1])[:, :, 4:, 5] = float("nan")
        assert torch.equal(lse, lse0)
        assert torch.equal(norm(out), norm(want)), (b, pos)


@pytest.mark.parametrize("D", [128, 64])
def test_pieces_without_weight(D):
    """A whole stretch of a long prefix weighs nothing beside the rest."""
    c = uniform(9000, [5, 40], 1, D, 2)
    sink(c.kp[:, 0, :4000], -512.0)
    base, lse0 = c.run()
    c.vp[0, 0, 7, 5] = INF
    out, lse = c.run()
    base[:, :, :4, 5] = float("nan")
    assert torch.equal(lse, lse0)
    assert torch.equal(torch.nan_to_num(out, 77., 88., 99.),
                       torch.nan_to_num(base, 77., 88., 99.))
