"""Token log probabilities, entropy, alternatives and their gradient on the GPU
vs the oracle.

Tolerances.  With R = max |s| over a row's finite s = z log2(e) / T:

* log2(e) / T carries two float32 roundings and s - m one, each at most 2^-24 of
  at most 2 R: the exponent of a term is off by at most 3 * 2^-23 R, taken as
  2^-21 R, and so are ln p and the normaliser;
* a thread adds at most V / 256 + 8 terms and then joins 8 levels of 2 roundings
  and one exponential (2^-22) each: a relative error of the sum of at most
  e = (V / 256 + 64) 2^-24 + 8 * 2^-21;
* the entropy is ln 2 (log2 S - A / S): A's terms weigh |s - m|, whose mean is
  at most E + log2 V for E the distance a reference may lie from the maximum
  (10) plus the mean distance from it: (2 log2 V + 24) e, and 2^-21 R as above
  times the spread of s, at most (2 log2 V + 24).

Gradient: p is off by a relative 2^-20 R + 2^-20 (exponent as above with the
normaliser's own float32 rounding, times ln 2, and the exponential); the sums of
given gradients by n 2^-24; the output's rounding by eps / 2 of its value (2^-8
in bf16).
"""

import numpy as np
import pytest
import torch

from oracle import logprobs as oracle
from tests._parity import lib_ready

pytestmark = pytest.mark.gpu
LOG2E = 1.4426950408889634


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def api():
    from speculative_decoding_verification_tree_gb300 import api as a
    return a


def np64(t):
    return t.detach().double().cpu().numpy()


def make(M, V, dtype, seed=0, std=2.5, pad=0, masked=0.0):
    """[M, V] logits as a view of rows padded by `pad` NaN logits."""
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(M, V + pad)) * std
    z[:, :V][rng.random((M, V)) < masked] = -np.inf
    z[:, V:] = np.nan
    return torch.from_numpy(z).to(dtype).cuda()[:, :V]


def spread(z, T):
    f = np.where(np.isfinite(z), np.abs(z), 0.0).max(-1)
    return f * LOG2E / T


def check(z, tokens, r, T, top, rows=None):
    zz = np64(z)
    M, V = zz.shape
    lp, lse, H, ids, tl = oracle.token_logprobs(zz, tokens, T, top)
    R = spread(zz, T)
    e = (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -18
    tol = (2.0 ** -21 * R + e)[:, None]
    assert (np.abs(np64(r.logprob).reshape(lp.shape) - lp) <= tol).all()
    assert (np.abs(np64(r.lse) - lse) <= tol[:, 0] * 1.5).all()
    if r.entropy is not None:
        w = 2 * np.log2(max(V, 2)) + 24
        assert (np.abs(np64(r.entropy) - H) <= w * tol[:, 0]).all()
    if top:
        assert np.array_equal(r.top_ids.cpu().numpy(), ids)
        fin = np.isfinite(tl)
        got = np64(r.top_logprob)
        assert np.array_equal(got[~fin], tl[~fin])
        assert (np.abs(got - np.where(fin, tl, 0))[fin]
                <= np.broadcast_to(tol, tl.shape)[fin]).all()


SHAPES = [(1, 1), (1, 2), (3, 7), (5, 100), (1, 1003), (33, 1000), (2, 4097),
          (7, 50257), (1, 128256), (400, 3001), (2, 151936)]


@pytest.mark.parametrize("M,V", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs(M, V, dtype):
    rng = np.random.default_rng(M + V)
    for T, n, top, pad, ent in ((1.0, 1, 0, 0, True), (0.7, 3, 5, 3, False),
                                (1.3, 2, 20, 8, True), (1.0, 0, 128, 1, True)):
        top = min(top, V)
        z = make(M, V, dtype, seed=V + n, pad=pad, masked=0.05 if V > 50 else 0)
        tok = rng.integers(-1, V, size=(M, n))
        zz = np64(z)
        # a masked token's log probability is -inf: not compared by difference
        for i in range(M):
            for j in range(n):
                if tok[i, j] >= 0 and np.isneginf(zz[i, tok[i, j]]):
                    tok[i, j] = int(np.argmax(zz[i]))
        r = api().spec_token_logprobs(z, torch.from_numpy(tok).int().cuda(),
                                      temperature=T, top=top, entropy=ent)
        assert (r.entropy is None) == (not ent)
        check(z, tok, r, T, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1000, 50257, 128256])
def test_ties_and_masked_vocabularies(V, dtype):
    """Constant rows, rows with fewer finite logits than alternatives, rows of
    two values, zeros of both signs: lower index first."""
    rng = np.random.default_rng(V)
    z = np.full((7, V), -1.0)
    z[1] = np.where(rng.random(V) < 0.5, 1.0, 2.0)
    z[2] = -np.inf
    z[2, rng.choice(V, 5, replace=False)] = rng.normal(size=5)
    z[3] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    z[4] = -np.inf
    z[4, V - 1] = 3.0
    z[5] = np.arange(V)[::-1] // 3 * 2.0 ** -10
    z[6] = torch.finfo(dtype).min
    z[6, ::17] = rng.normal(size=len(z[6, ::17]))
    z = torch.from_numpy(z).to(dtype).cuda()
    zz = np64(z)
    tok = zz.argmax(-1)[:, None]
    r = api().spec_token_logprobs(z, torch.from_numpy(tok).int().cuda(),
                                  top=20, entropy=True)
    keep = [0, 1, 2, 3, 4, 5]
    pick = lambda t: t[keep]
    check(z[keep], tok[keep], type(r)(*map(pick, r)), 1.0, 20)
    # lowest-value masks: s = -3e38 log2(e) overflows to probability 0
    assert np.array_equal(r.top_ids[6].cpu().numpy(), oracle.token_logprobs(
        zz[6:], tok[6:], 1.0, 20)[3][0])
    lp = oracle.log_softmax(np.where(zz[6:] < -1e30, -np.inf, zz[6:]), 1.0)[0]
    assert abs(float(r.logprob[6, 0]) - lp.max()) < 1e-4
    assert np.isfinite(float(r.entropy[6]))


def test_rows_are_picked_repeated_and_absent():
    z = make(9, 4001, torch.bfloat16, seed=3)
    rows = np.array([[4, 4, -1], [8, 0, 9], [1, 2, 3]])
    rng = np.random.default_rng(1)
    tok = rng.integers(0, 4001, size=(3, 3))
    r = api().spec_token_logprobs(
        z.reshape(3, 3, 4001), torch.from_numpy(tok).int().cuda(), top=4,
        entropy=True, rows=torch.from_numpy(rows).int().cuda())
    assert r.logprob.shape == (3, 3) and r.top_ids.shape == (3, 3, 4)
    ok = (rows >= 0) & (rows < 9)
    sel = torch.from_numpy(rows[ok]).cuda()
    flat = type(r)(*[x[torch.from_numpy(ok).cuda()] for x in r])
    check(z[sel], tok[ok][:, None], flat, 1.0, 4)
    for x, absent in ((r.logprob, 0), (r.lse, 0), (r.entropy, 0),
                      (r.top_ids, -1), (r.top_logprob, 0)):
        assert (x[torch.from_numpy(~ok).cuda()] == absent).all()


def test_nan_and_infinite_rows():
    z = make(5, 3001, torch.float32, seed=5)
    z[1, 77] = float("nan")
    z[2, 5] = float("inf")
    z[3] = float("-inf")
    z[4] = float("nan")
    tok = torch.full((5,), 100, dtype=torch.int32, device="cuda")
    r = api().spec_token_logprobs(z, tok, top=6, entropy=True)
    assert torch.isfinite(r.logprob[0]) and torch.isfinite(r.entropy[0])
    assert torch.isnan(r.logprob[1:]).all() and torch.isnan(r.entropy[1:]).all()
    zz = np64(z)
    zz[1, 77] = -1e9
    assert r.top_ids[1].tolist() == np.argsort(-zz[1], kind="stable")[:6].tolist()
    assert int(r.top_ids[2, 0]) == 5
    assert r.top_ids[3].tolist() == [0, 1, 2, 3, 4, 5]
    assert (r.top_ids[4] == -1).all() and torch.isnan(r.top_logprob[4]).all()
    g = api().spec_token_logprobs_grad(z, tok, r.lse, torch.ones(5).cuda())
    assert torch.isfinite(g[0]).all() and torch.isnan(g[1:]).all()


def grad_tol(z, tok, g, gh, T, dtype, want):
    lp, _ = oracle.log_softmax(z, T)
    p = np.exp(lp)
    V = z.shape[1]
    ga = np.abs(np.where((tok >= 0) & (tok < V), g, 0)).sum(-1, keepdims=True)
    R = spread(z, T)[:, None]
    w = ga.copy()
    if gh is not None:
        H = -np.where(p > 0, p * np.where(p > 0, lp, 0), 0).sum(-1, keepdims=True)
        w = w + np.abs(gh)[:, None] * (np.abs(np.where(p > 0, lp, 0)) + H + 1)
    tol = p * w * (2.0 ** -20 * (R + 2) + tok.shape[1] * 2.0 ** -24) / T
    for i in range(len(tok)):
        for x in tok[i]:
            if 0 <= x < V:
                tol[i, x] += ga[i, 0] * (2.0 ** -23 * (tok.shape[1] + 2)) / T
    return tol + torch.finfo(dtype).eps / 2 * np.abs(want) + 1e-38


@pytest.mark.parametrize("M,V", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient(M, V, dtype):
    rng = np.random.default_rng(M * V + 1)
    for T, n, top, pad, ent, where in (
            (1.0, 1, 0, 0, False, "new"), (0.7, 3, 5, 3, True, "new"),
            (1.3, 64, 0, 8, True, "same"), (1.0, 0, 3, 1, True, "strided")):
        top = min(top, V)
        z = make(M, V, dtype, seed=V + n, pad=pad, masked=0.05 if V > 50 else 0)
        zz = np64(z)
        tok = rng.integers(-1, V, size=(M, n))
        if n > 1:
            tok[:, n - 1] = tok[:, 0]          # the same token twice
        g = rng.normal(size=(M, n)).astype(np.float32)
        gh = rng.normal(size=M).astype(np.float32) if ent else None
        t32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
        r = api().spec_token_logprobs(z, t32(tok).int(), temperature=T, top=top,
                                      entropy=ent)
        # unequal to the forward's choice: the alternatives are given tokens
        ids = rng.integers(0, V, size=(M, top))
        gt = rng.normal(size=(M, top)).astype(np.float32)
        kw = dict(temperature=T)
        if ent:
            kw.update(entropy=r.entropy, g_entropy=t32(gh))
        if top:
            kw.update(top_ids=t32(ids).int(), g_top=t32(gt))
        out = None
        if where == "same":
            out = z
        elif where == "strided":
            out = torch.full((M, V + 5), 7.0, dtype=dtype, device="cuda")[:, :V]
        d = api().spec_token_logprobs_grad(z, t32(tok).int(), r.lse, t32(g),
                                           out=out, **kw)
        alltok = np.concatenate([tok, ids], 1)
        allg = np.concatenate([g, gt], 1).astype(np.float64)
        want = oracle.grad(zz, alltok, allg, gh, T)
        tol = grad_tol(zz, alltok, allg, gh, T, dtype, want)
        bad = np.abs(np64(d) - want) > tol
        assert not bad.any(), (T, n, where, np.argwhere(bad)[:5])
        if where == "strided":
            buf = torch.as_strided(out, (M, V + 5), (V + 5, 1))
            assert (buf[:, V:] == 7).all()


def test_gradient_against_differences():
    """Central differences of the GPU's own forward values.  Their error: h^2/6
    times a third derivative of at most 2 (|g| + |g_H| (ln V + 2)) per unit of
    gradient, and float32 values (of magnitude below 8) over 2h."""
    M, V, h = 1, 37, 2.0 ** -4
    z = make(M, V, torch.float32, seed=11, std=1.0)
    tok = torch.tensor([[3, 20, 3]], dtype=torch.int32, device="cuda")
    g, gh = [0.5, -1.25, 0.75], -0.5
    gv = torch.tensor([g], device="cuda")

    def value(x):
        r = api().spec_token_logprobs(x, tok, entropy=True)
        return (np64(r.logprob) * g).sum(-1) + gh * np64(r.entropy)
    r = api().spec_token_logprobs(z, tok, entropy=True)
    d = np64(api().spec_token_logprobs_grad(
        z, tok, r.lse, gv, entropy=r.entropy,
        g_entropy=torch.tensor([gh], device="cuda")))[0]
    eye = torch.eye(V, device="cuda") * h
    t2 = tok.expand(V, 3).contiguous()

    def values(x):
        r = api().spec_token_logprobs(x, t2, entropy=True)
        return (np64(r.logprob) * g).sum(-1) + gh * np64(r.entropy)
    num = (values(z + eye) - values(z - eye)) / (2 * h)
    tol = h * h / 6 * 2 * (2.5 + 0.5 * (np.log(V) + 2)) + 8 * 4 * 2.0 ** -23 / h
    assert np.abs(num - d).max() <= tol


def test_far_rows_pass_32_bits():
    """Row offsets past 2^31 elements (bf16 rows 2^27 elements apart)."""
    ld, V = 1 << 27, 2000
    buf = torch.empty(17 * ld + V, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(buf, (18, V), (ld, 1))
    z.copy_(make(18, V, torch.bfloat16, seed=2))
    tok = torch.randint(V, (18, 1), device="cuda").int()
    r = api().spec_token_logprobs(z, tok, top=3, entropy=True)
    zc = z.contiguous()
    check(zc, tok.cpu().numpy(), r, 1.0, 3)
    want = api().spec_token_logprobs_grad(zc, tok, r.lse,
                                          torch.ones(18, 1).cuda())
    got = api().spec_token_logprobs_grad(z, tok, r.lse,
                                         torch.ones(18, 1).cuda(), out=z)
    assert torch.equal(got, want)


def test_streams_and_graphs():
    """A call on another stream, and one captured and replayed on new inputs."""
    M, V = 40, 32000
    z = make(M, V, torch.bfloat16, seed=1)
    tok = torch.randint(V, (M, 1), device="cuda").int()
    g = torch.randn(M, 1, device="cuda")

    def both():
        r = api().spec_token_logprobs(z, tok, top=5, entropy=True)
        d = api().spec_token_logprobs_grad(z, tok, r.lse, g,
                                           entropy=r.entropy, g_entropy=g[:, 0]
                                           .contiguous())
        return tuple(r) + (d,)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = both()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for x, y in zip(both(), other):
        assert torch.equal(x, y)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = both()
    z.copy_(make(M, V, torch.bfloat16, seed=2))
    gr.replay()
    for x, y in zip(both(), out):
        assert torch.equal(x, y)
