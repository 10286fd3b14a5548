"""Gradient of log probabilities and entropies for rows with large finite logits
or at very low temperatures, against the oracle.

Tolerances, with the notation and the tolerance ts of log2 S of
test_gpu_logprobs_masks.py:

* ln p is off by r = 2^-21 (q + |d| + 60) + 1.5 ts: the scaled distance's five
  roundings, and the normaliser's.  q = |z| log2(e) / T + |lse| where p is formed
  from the given float32 normaliser, which is below 2^12; 0 elsewhere (there the
  row's terms are formed again).  p is off by that factor, the logarithm in the
  entropy's part by that amount, the entropy by its own tolerance;
* sums of n given gradients: n 2^-24 of their magnitudes; 1 / T and the products:
  2^-22; the output's rounding: eps / 2 of its value; exponentials below 2^-126
  are 0.
"""

import numpy as np
import pytest
import torch

from oracle import logprobs as oracle
from tests._parity import lib_ready
from tests.test_gpu_logprobs import api, np64
from tests.test_gpu_logprobs_masks import LOG2E, MASKS, masked_rows, terms

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def run(z, T, n, top, ent, where, seed=0):
    """The gradient of a forward pass's outputs, checked."""
    zz, dtype = np64(z), z.dtype
    M, V = zz.shape
    rng = np.random.default_rng(seed)
    t32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    tok = rng.integers(-1, V, size=(M, n))
    if n > 2:
        tok[:, 1], tok[:, 2] = 0, np64(z).argmax(-1)
        tok[:, n - 1] = tok[:, 0]
    g = rng.normal(size=(M, n)).astype(np.float32)
    gh = rng.normal(size=M).astype(np.float32) if ent else None
    gt = rng.normal(size=(M, top)).astype(np.float32)
    r = api().spec_token_logprobs(z, t32(tok).int(), temperature=T, top=top,
                                  entropy=ent)
    kw = dict(temperature=T)
    if ent:
        kw.update(entropy=r.entropy, g_entropy=t32(gh))
    if top:
        kw.update(top_ids=r.top_ids, g_top=t32(gt))
        tok = np.concatenate([tok, r.top_ids.cpu().numpy()], 1)
        g = np.concatenate([g, gt], 1)
    out = None
    if where == "same":
        out = z
    elif where == "strided":
        out = torch.full((M, V + 5), 7.0, dtype=dtype, device="cuda")[:, :V]
    got = np64(api().spec_token_logprobs_grad(
        z, t32(tok[:, :n]).int(), r.lse, t32(g[:, :n]), out=out, **kw))
    if where == "strided":
        buf = torch.as_strided(out, (M, V + 5), (V + 5, 1))
        assert (buf[:, V:] == 7).all()

    g = g.astype(np.float64)
    want = oracle.grad(zz, tok, g, gh, T)
    lp, lse, H, _, _ = oracle.token_logprobs(zz, tok, T, 0)
    d, p, ad, E, e, ts = terms(zz, T)
    lse = np.abs(lse)[:, None]
    az = np.where(np.isfinite(zz), np.abs(zz), 0) * LOG2E / T
    q = np.where(lse < 4096, np.where(p > 0, az, 0) + lse, 0)
    rel = 2.0 ** -21 * (q + ad + 60) + 1.5 * ts[:, None]
    ok = (tok >= 0) & (tok < V)
    ga = np.where(ok, np.abs(g), 0).sum(-1)
    w = np.broadcast_to(ga[:, None], p.shape).copy()
    ag = np.zeros_like(w)
    if ent:
        ag = np.abs(gh.astype(np.float64))[:, None]
        w = w + ag * (ad + H[:, None] + 1)
    W = (p * (ad + 10) ** 2).sum(-1)
    th = (2.0 ** -20 * W + 4 * e * (E + 20))[:, None]
    tol = p * (rel * w + ag * (rel + th) + tok.shape[1] * 2.0 ** -24 * w)
    for i in range(M):
        for x in tok[i][ok[i]]:
            tol[i, x] += ga[i] * 2.0 ** -22 * (tok.shape[1] + 2)
    tol = ((tol + 2.0 ** -125 * (w + 1)) / T
           + (torch.finfo(dtype).eps / 2 + 2.0 ** -22) * np.abs(want))
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (T, n, where, np.argwhere(bad)[:4], got[bad][:4],
                           want[bad][:4])


@pytest.mark.parametrize("mask", MASKS, ids=str)
@pytest.mark.parametrize("T", [0.6, 1.0, 2.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_finite_masks(mask, T, dtype):
    for V, pad, n, top, ent, where in ((1003, 3, 3, 0, True, "new"),
                                       (9000, 8, 4, 5, True, "same"),
                                       (20011, 1, 64, 3, False, "same"),
                                       (9001, 7, 1, 0, True, "strided")):
        run(masked_rows(V, dtype, mask, pad, seed=V), T, n, top, ent, where,
            seed=V)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1e-9, 1e-6, 1e-3, 1e6])
def test_far_temperatures(T, dtype):
    for V, where in ((17000, "same"), (1003, "strided")):
        rng = np.random.default_rng(V)
        z = rng.normal(size=(6, V)) * 8
        z[0, :V // 2] = -1e9
        z[1] = np.round(z[1])
        z = torch.from_numpy(z).to(dtype).cuda()
        run(z, T, 3, 2, True, where, seed=V)


def test_masked_rows_without_a_gradient_stay_zero():
    """A row that is masked off with a finite value and given no gradient, as in
    a padded batch, adds none."""
    for dtype in (torch.float32, torch.bfloat16):
        for value in (-1e9, -1e30, torch.finfo(dtype).min):
            z = torch.full((3, 9000), value, dtype=dtype, device="cuda")
            z[1] = torch.randn(9000, device="cuda")
            tok = torch.full((3,), 5, dtype=torch.int32, device="cuda")
            r = api().spec_token_logprobs(z, tok, entropy=True)
            zero, one = torch.zeros(3).cuda(), torch.zeros(3).cuda()
            one[1] = 1
            d = api().spec_token_logprobs_grad(z, tok, r.lse, one)
            assert (d[[0, 2]] == 0).all() and d[1].abs().sum() > 0
            d = api().spec_token_logprobs_grad(
                z, tok, r.lse, one, entropy=r.entropy, g_entropy=zero)
            assert (d[[0, 2]] == 0).all()
