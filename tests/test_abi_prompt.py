"""Refusals of the prompt attention (no device work), and its oracle against
scaled dot products with a causal mask."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import prompt as oracle
from speculative_decoding_verification_tree_gb300 import _lib, api

FAKE = ctypes.c_void_p(0x7f0000000000)  # never dereferenced: calls fail early
ODD = ctypes.c_void_p(0x7f0000000008)   # 8-byte aligned only
ODD2 = ctypes.c_void_p(0x7f0000000002)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    _lib.load()
    return _lib


def test_argument_errors(lib):
    def call(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, st=FAKE, B=2, T=9,
             Hq=8, Hkv=2, D=128, scale=0.1, out=FAKE, lse=None):
        return lib.raw("spec_prompt_attention", q, qs, k, ks, v, vs, st, B, T,
                       Hq, Hkv, D, scale, out, lse, None)
    for kw in (dict(B=-1), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=7),
               dict(Hq=258, qs=1 << 20), dict(T=(1 << 30) + 1), dict(qs=1016),
               dict(ks=248), dict(vs=128), dict(qs=1 << 38)):
        assert call(**kw) == lib.SPEC_ERR_SHAPE, kw
    for kw in (dict(D=32), dict(D=96), dict(D=256), dict(qs=1028),
               dict(ks=260), dict(vs=257)):
        assert call(**kw) == lib.SPEC_ERR_UNSUPPORTED, kw
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(q=None), dict(k=None),
               dict(v=None), dict(st=None), dict(out=None), dict(q=ODD),
               dict(k=ODD), dict(v=ODD), dict(out=ODD), dict(st=ODD2),
               dict(lse=ODD2)):
        assert call(**kw) == lib.SPEC_ERR_ARG, kw
    assert call(B=0, q=None, st=None) == lib.SPEC_OK
    assert call(T=0, q=None, out=None) == lib.SPEC_OK


def test_wrapper_refuses(monkeypatch):
    monkeypatch.setattr(_lib, "call", lambda *a: pytest.fail("called"))
    monkeypatch.setattr(api, "_index", lambda t: -1)  # CPU tensors pass
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    q, k, st = b(9, 8, 128), b(9, 2, 128), torch.zeros(3, dtype=torch.int32)
    f = api.spec_prompt_attention
    bad = [lambda: f(q.float(), k, k, st), lambda: f(q, k, k, st.long()),
           lambda: f(q, k[:8], k, st), lambda: f(q, k, b(9, 2, 64), st),
           lambda: f(q, k, b(9, 4, 128)[:, ::2], st),
           lambda: f(q, k, b(2, 9, 128).transpose(0, 1), st),
           lambda: f(q, k, k, st[:0]), lambda: f(q, k, k, st, out=q[:8]),
           lambda: f(q, k, k, st, out=q, lse=torch.zeros(9, 7))]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_oracle_equals_causal_attention():
    rng = np.random.default_rng(0)
    q, k, v = (rng.normal(size=(12, h, 8)) for h in (4, 2, 2))
    out, lse, _, _ = oracle.prompt_attention(q, k, v, [1, 6, 6, 11], 0.3)
    assert np.isnan(out[[0, 11]]).all()
    t = lambda x: torch.from_numpy(x)
    for a, z in ((1, 6), (6, 11)):
        want = torch.nn.functional.scaled_dot_product_attention(
            t(q[a:z]).transpose(0, 1), t(k[a:z].repeat(2, 1)).transpose(0, 1),
            t(v[a:z].repeat(2, 1)).transpose(0, 1), is_causal=True, scale=0.3)
        assert np.allclose(out[a:z], want.transpose(0, 1).numpy())
        s = 0.3 * np.einsum("ihd,jhd->hij", q[a:z], k[a:z].repeat(2, 1))
        s[:, np.triu(np.ones((5, 5), bool), 1)] = -np.inf
        assert np.allclose(lse[a:z], np.log2(np.exp(s).sum(-1)).T)
