"""Token log probabilities, entropy and alternatives of rows that hold large
finite values (masks that are not -inf), against the oracle.

Tolerances, with d = (z - max z) log2(e) / T in base 2, p the probabilities and
E = sum p |d|:

* a distance is a float32 difference times a float32 factor that carries three
  roundings (the temperature's, log2(e)'s, the quotient's): off by 5 * 2^-24 of
  itself.  References lie at most 10 below the maxima of what they stand for, and
  moving one adds distances of that kind: an exponent is off by at most
  2^-21 (|d| + 10), which reaches log2 S weighted by p: 2^-21 (E + 10);
* sums: e = (V / 256 + 64) 2^-24 + 2^-18, as in test_gpu_logprobs.py;
* ln p(t): both, and 2^-21 (|d_t| + 10) for the token's own distance;
* the normaliser (base 2): both times log2(e), and 2^-22 (|lse| + 40) for the
  maximum times the factor (four roundings);
* the entropy: ln 2 (log2 S - A / S), A's terms p |d| off by the exponent's error
  and the distance's, together below 2^-20 sum p (|d| + 10)^2, and the sums' and
  joins' roundings, 4 e (E + 20).

Values past float32's range are infinite.
"""

import numpy as np
import pytest
import torch

from oracle import logprobs as oracle
from tests._parity import lib_ready
from tests.test_gpu_logprobs import api, np64

pytestmark = pytest.mark.gpu
LOG2E = 1.4426950408889634
MASKS = [-1e4, -1e9, -1e10, -1e20, -1e30, -1e38, "lowest"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def masked_rows(V, dtype, mask, pad=0, seed=0, repeat=1):
    """Rows with `mask` in many places, inside rows padded with NaN."""
    rng = np.random.default_rng(seed)
    m = torch.finfo(dtype).min if mask == "lowest" else mask
    n = 10 * repeat
    z = rng.normal(size=(n, V + pad)) * 2.5
    for a in range(0, n, 10):
        z[a, :64] = m                       # a thread's first logits, and more
        z[a + 1, rng.random(V + pad) < 31 / 32] = m
        z[a + 2, 0] = m                     # a logit before the 16-byte groups
        z[a + 3, V - 1] = m                 # and one behind them
        z[a + 4] = m
        z[a + 4, V // 2] = 1.0              # one survivor
        z[a + 5] = m                        # none
        z[a + 6, rng.random(V + pad) < 0.5] = m
        z[a + 6, rng.random(V + pad) < 0.3] = -np.inf
        z[a + 7, :V // 2] = m
        z[a + 8, V // 3:] = m
        z[a + 9, rng.random(V + pad) < 0.2] = m
        z[a + 9] *= -1                      # large positive ones
    z[:, V:] = np.nan
    return torch.from_numpy(z).to(dtype).cuda()[:, :V]


def rounded(x):
    """Float64 values with those past float32's range infinite."""
    with np.errstate(over="ignore"):
        return np.where(np.isinf(x.astype(np.float32)),
                        x.astype(np.float32).astype(np.float64), x)


def close(got, want, tol, what):
    want = rounded(want)
    tol = np.broadcast_to(tol, want.shape)
    same = np.isinf(want) & (got == want)
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= tol))
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4],
                           want[bad][:4])


def terms(z, T):
    """d, p, E and the tolerance of log2 S."""
    V = z.shape[-1]
    d = (z - z.max(-1, keepdims=True)) * LOG2E / T
    p = 2.0 ** d / (2.0 ** d).sum(-1, keepdims=True)
    ad = np.where(p > 0, np.abs(np.where(p > 0, d, 0)), 0)
    E = (p * ad).sum(-1)
    e = (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -18
    return d, p, ad, E, e, 2.0 ** -21 * (E + 10) + e


def check(z, tok, r, T, top):
    zz = np64(z)
    lp, lse, H, ids, tl = oracle.token_logprobs(zz, tok, T, top)
    d, p, ad, E, e, ts = terms(zz, T)
    at = np.clip(tok, 0, None)
    own = np.abs(np.take_along_axis(d, at, 1))
    own = np.where(np.isfinite(own), own, 0)
    close(np64(r.logprob), lp, ts[:, None] + 2.0 ** -21 * (own + 10), "logprob")
    close(np64(r.lse), lse, 1.4427 * ts + 2.0 ** -22 * (np.abs(lse) + 40), "lse")
    if r.entropy is not None:
        W = (p * (ad + 10) ** 2).sum(-1)
        close(np64(r.entropy), H, 2.0 ** -20 * W + 4 * e * (E + 20), "entropy")
    if top:
        assert np.array_equal(r.top_ids.cpu().numpy(), ids)
        own = np.abs(np.take_along_axis(d, ids, 1))
        own = np.where(np.isfinite(own), own, 0)
        close(np64(r.top_logprob), tl, ts[:, None] + 2.0 ** -21 * (own + 10),
              "top")


@pytest.mark.parametrize("mask", MASKS, ids=str)
@pytest.mark.parametrize("T", [0.6, 1.0, 1.5, 2.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_finite_masks(mask, T, dtype):
    for V, pad, top, ent, rep in ((32000, 0, 0, True, 1),     # clusters
                                  (32000, 0, 20, False, 1),
                                  (1003, 3, 5, True, 1),
                                  (4001, 7, 40, True, 31)):   # a CTA a row
        z = masked_rows(V, dtype, mask, pad, seed=V, repeat=rep)
        rng = np.random.default_rng(V + 1)
        tok = rng.integers(0, V, size=(len(z), 4))
        tok[:, 1], tok[:, 2] = 0, V - 1
        tok[:, 3] = np64(z).argmax(-1)
        tok[::3, 0] = -1
        r = api().spec_token_logprobs(z, torch.from_numpy(tok).int().cuda(),
                                      temperature=T, top=top, entropy=ent)
        check(z, tok, r, T, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1e-9, 1e-6, 1e-3, 300.0, 1e6, 1e9])
def test_far_temperatures(T, dtype):
    """Ordinary logits whose scaled values are as large as masked ones, and
    masks that a high temperature brings back into view."""
    for V, M in ((32000, 3), (1003, 40)):
        rng = np.random.default_rng(V)
        z = rng.normal(size=(M, V)) * 8
        z[0, :V // 2] = -1e9
        z = torch.from_numpy(z).to(dtype).cuda()
        tok = np.stack([np64(z).argmax(-1), np.arange(M) * 7], 1)
        r = api().spec_token_logprobs(z, torch.from_numpy(tok).int().cuda(),
                                      temperature=T, top=3, entropy=True)
        check(z, tok, r, T, 3)


def test_rows_of_lowest_values_only():
    """A row whose mask leaves nothing, with a finite mask, is uniform."""
    for dtype in (torch.float32, torch.bfloat16):
        for V in (7, 4096, 50257):
            z = torch.full((2, V), torch.finfo(dtype).min, dtype=dtype,
                           device="cuda")
            tok = torch.tensor([0, V - 1], dtype=torch.int32, device="cuda")
            r = api().spec_token_logprobs(z, tok, top=2, entropy=True)
            n = np.log(V)
            # V / 256 + 64 additions of ones, a logarithm: 2^-22 of it and e
            tol = 2.0 ** -21 * n + (V / 256 + 64) * 2.0 ** -24
            assert (np.abs(np64(r.logprob) + n) <= tol).all()
            assert (np.abs(np64(r.entropy) - n) <= tol).all()
            assert r.top_ids.tolist() == [[0, 1], [0, 1]]
