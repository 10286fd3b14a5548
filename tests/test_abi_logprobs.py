"""Refusals of the log-probability entry points (no device work), and the
oracle's gradient against differences."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import logprobs as oracle
from speculative_decoding_verification_tree_gb300 import _lib, api

FAKE = ctypes.c_void_p(0x7f0000000000)  # never dereferenced: calls fail early
ODD = ctypes.c_void_p(0x7f0000000001)
ODD2 = ctypes.c_void_p(0x7f0000000002)
FAR = ctypes.c_void_p(0x7f4000000000)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    _lib.load()
    return _lib


def test_forward_argument_errors(lib):
    def call(z=FAKE, dt=1, ld=100, R=4, V=100, rows=None, M=4, tok=FAKE, n=2,
             top=3, T=1.0, lp=FAKE, lse=FAKE, ent=None, ids=FAKE, tl=FAKE):
        return lib.raw("spec_token_logprobs", z, dt, ld, R, V, rows, M, tok, n,
                       top, T, lp, lse, ent, ids, tl, None)
    for dt in (-1, 2):
        assert call(dt=dt) == lib.SPEC_ERR_DTYPE
    for kw in (dict(R=-1), dict(M=-1), dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25),
               dict(ld=99), dict(n=-1), dict(n=65), dict(top=-1), dict(top=129,
               V=200, ld=200), dict(top=101), dict(M=5), dict(M=1 << 28,
               R=1 << 28)):
        assert call(**kw) == lib.SPEC_ERR_SHAPE, kw
    for kw in (dict(T=0.0), dict(T=-1.0), dict(T=float("nan")),
               dict(T=float("inf")), dict(z=None), dict(tok=None),
               dict(lp=None), dict(ids=None), dict(tl=None), dict(z=ODD),
               dict(z=ODD2, dt=0), dict(rows=ODD2), dict(tok=ODD2),
               dict(lp=ODD2), dict(lse=ODD2), dict(ent=ODD2), dict(ids=ODD2),
               dict(tl=ODD2)):
        assert call(**kw) == lib.SPEC_ERR_ARG, kw
    assert call(M=0, z=None, tok=None, lp=None) == lib.SPEC_OK


def test_gradient_argument_errors(lib):
    def call(z=FAKE, dt=1, ld=100, M=4, V=100, tok=FAKE, n=2, ids=None, top=0,
             T=1.0, lse=FAKE, ent=None, g=FAKE, gt=None, gh=None, d=FAR,
             ldd=100):
        return lib.raw("spec_token_logprobs_grad", z, dt, ld, M, V, tok, n, ids,
                       top, T, lse, ent, g, gt, gh, d, ldd, None)
    assert call(dt=7) == lib.SPEC_ERR_DTYPE
    for kw in (dict(M=-1), dict(V=0), dict(ld=99), dict(ldd=99), dict(n=65),
               dict(n=-1), dict(top=129), dict(top=-1),
               dict(M=(1 << 31) - 1, V=20000, ld=20000, ldd=20000)):
        assert call(**kw) == lib.SPEC_ERR_SHAPE, kw
    over = ctypes.c_void_p(FAKE.value + 2)
    for kw in (dict(T=0.0), dict(z=None), dict(d=None), dict(lse=None),
               dict(tok=None), dict(g=None), dict(top=1), dict(top=1, ids=FAKE),
               dict(ent=FAKE), dict(gh=FAKE), dict(z=ODD), dict(d=ODD),
               dict(lse=ODD2), dict(g=ODD2), dict(d=over),
               dict(d=FAKE, ldd=120)):
        assert call(**kw) == lib.SPEC_ERR_ARG, kw
    assert call(M=0, z=None, d=None) == lib.SPEC_OK


def test_wrappers_refuse(monkeypatch):
    """Shapes, dtypes and strides that do not fit, before any library call."""
    monkeypatch.setattr(_lib, "call", lambda *a: pytest.fail("called"))
    monkeypatch.setattr(api, "_index", lambda t: -1)  # CPU tensors pass
    z = torch.zeros(4, 10)
    tok = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(4)
    bad = [
        lambda: api.spec_token_logprobs(z.half(), tok),
        lambda: api.spec_token_logprobs(z, tok.long()),
        lambda: api.spec_token_logprobs(z, tok[:3]),
        lambda: api.spec_token_logprobs(z.T, torch.zeros(10,
                                        dtype=torch.int32)),
        lambda: api.spec_token_logprobs(torch.zeros(4, 3, 10)[:, :2],
                                        torch.zeros(4, 2, dtype=torch.int32)),
        lambda: api.spec_token_logprobs(z, tok, rows=tok.long()),
        lambda: api.spec_token_logprobs_grad(z, tok, f, f, entropy=f),
        lambda: api.spec_token_logprobs_grad(z, tok, f, f, g_top=f),
        lambda: api.spec_token_logprobs_grad(z, tok, f, f[:2]),
        lambda: api.spec_token_logprobs_grad(z, tok, f, f.double()),
        lambda: api.spec_token_logprobs_grad(z, tok, f, f,
                                             out=torch.zeros(4, 11)),
        lambda: api.spec_token_logprobs_grad(z, tok, f, f, out=z.bfloat16()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_cpu_tensors_are_refused():
    z = torch.zeros(4, 10)
    with pytest.raises(ValueError):
        api.spec_token_logprobs(z, torch.zeros(4, dtype=torch.int32))


def test_oracle_gradient_equals_differences():
    rng = np.random.default_rng(0)
    z = rng.normal(size=(2, 9))
    z[1, 4] = -np.inf
    tok = np.array([[2, 2, -1], [8, 0, 9]])
    g, gh, T = rng.normal(size=(2, 3)), rng.normal(size=2), 0.8

    def value(x):
        lp, _, H, _, _ = oracle.token_logprobs(x, tok, T)
        return (g * lp).sum() + (gh * H).sum()
    d = oracle.grad(z, tok, g, gh, T)
    assert d[1, 4] == 0
    for i in range(2):
        for x in range(9):
            if np.isinf(z[i, x]):
                continue
            e = np.zeros_like(z)
            e[i, x] = 1e-5
            num = (value(z + e) - value(z - e)) / 2e-5
            assert abs(num - d[i, x]) < 1e-8


def test_oracle_orders_alternatives_by_value_then_index():
    z = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0]])
    _, lse, H, ids, lp = oracle.token_logprobs(z, np.zeros((1, 0), int), 1.0, 4)
    assert ids.tolist() == [[1, 2, 4, 0]]
    p = np.exp(z - np.log(np.exp(z[z > -9]).sum()))
    assert np.allclose(np.exp(lp[0]), p[0][[1, 2, 4, 0]])
    assert np.isclose(lse[0], np.log2(np.exp(z[z > -9]).sum()))
    assert np.isclose(H[0], -(p[p > 0] * np.log(p[p > 0])).sum())
