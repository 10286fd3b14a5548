"""Refusals of the shared-prefix attention (no device work), and its oracle
against the one that knows no sharing."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import shared as oracle
from oracle.attention import tree_attention
from oracle.tree import tree_mask
from speculative_decoding_verification_tree_gb300 import _lib, api

FAKE = ctypes.c_void_p(0x7f0000000000)  # never dereferenced: calls fail early
ODD = ctypes.c_void_p(0x7f0000000008)   # 8-byte aligned only
ODD4 = ctypes.c_void_p(0x7f0000000004)
ODD2 = ctypes.c_void_p(0x7f0000000002)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    _lib.load()
    return _lib


def test_argument_errors(lib):
    size = lambda *a: lib.raw("spec_tree_attention_shared_workspace_bytes", *a)
    f = size(2, 8, 8, 2, 128, 1, 5000, 64)
    assert f > 0 and f % 256 == 0

    def call(q=FAKE, kp=FAKE, vp=FAKE, sl=FAKE, gs=FAKE, k=FAKE, v=FAKE,
             pre=FAKE, mb=FAKE, B=2, N=8, Hq=8, Hkv=2, D=128, g=1, Sp=5000,
             S=64, scale=0.1, out=FAKE, lse=None, ws=FAKE, nbytes=f):
        return lib.raw("spec_tree_attention_shared", q, kp, vp, sl, gs, k, v,
                       pre, mb, B, N, Hq, Hkv, D, g, Sp, S, scale, out, lse,
                       ws, nbytes, None)
    for kw in (dict(B=-1), dict(B=65536), dict(N=0), dict(N=65), dict(Hq=7),
               dict(Hq=0), dict(Hkv=0), dict(Hq=258), dict(g=0), dict(g=257),
               dict(Sp=-1), dict(Sp=(1 << 30) + 1), dict(S=7),
               dict(S=(1 << 30) + 1), dict(B=65535, Hq=1 << 16,
                                           Hkv=1 << 16)):
        assert call(**kw) == lib.SPEC_ERR_SHAPE, kw
        d = dict(B=2, N=8, Hq=8, Hkv=2, D=128, g=1, Sp=5000, S=64)
        d.update(kw)
        assert size(*d.values()) == 0
    for D in (0, 32, 96, 256):
        assert call(D=D) == lib.SPEC_ERR_UNSUPPORTED
        assert size(2, 8, 8, 2, D, 1, 5000, 64) == 0
    for kw in (dict(scale=0.0), dict(scale=float("nan")),
               dict(scale=float("inf")), *({n: None} for n in (
                   "q", "kp", "vp", "sl", "gs", "k", "v", "pre", "mb", "out")),
               *({n: ODD} for n in ("q", "kp", "vp", "k", "v", "out")),
               *({n: ODD2} for n in ("sl", "gs", "pre", "lse")), dict(mb=ODD4)):
        assert call(**kw) == lib.SPEC_ERR_ARG, kw
    for kw in (dict(ws=None), dict(ws=ODD), dict(nbytes=f - 1)):
        assert call(**kw) == lib.SPEC_ERR_WORKSPACE, kw
    # without shared positions their arrays may be missing (here the call then
    # stops at the workspace)
    assert call(Sp=0, kp=None, vp=None, ws=None) == lib.SPEC_ERR_WORKSPACE
    assert call(B=0, q=None, ws=None, nbytes=0) == lib.SPEC_OK
    assert size(0, 8, 8, 2, 128, 1, 5000, 64) == 0


def test_wrapper_refuses(monkeypatch):
    monkeypatch.setattr(_lib, "call", lambda *a: pytest.fail("called"))
    monkeypatch.setattr(api, "_index", lambda t: -1)  # CPU tensors pass
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    good = dict(q=b(2, 3, 8, 64), kp=b(1, 2, 20, 64), vp=b(1, 2, 20, 64),
                sl=i(1), gs=i(2), k=b(2, 2, 9, 64), v=b(2, 2, 9, 64), pre=i(2),
                mb=torch.zeros(2, 3, dtype=torch.int64))
    bad = dict(q=good["q"].float(), kp=b(1, 4, 20, 64), vp=b(1, 2, 21, 64),
               sl=i(2), gs=i(1), k=b(2, 2, 64, 9).transpose(2, 3),
               v=b(2, 2, 10, 64), pre=i(2).long(), mb=i(2, 3))
    for name, t in bad.items():
        with pytest.raises(ValueError):
            api.spec_tree_attention_shared(*dict(good, **{name: t}).values())
    for kw in (dict(out=b(2, 3, 8, 128)), dict(lse=torch.zeros(2, 3, 7)),
               dict(ws=torch.zeros(9))):
        kw.setdefault("ws", torch.zeros(9, dtype=torch.uint8))
        kw.setdefault("out", b(2, 3, 8, 64))
        with pytest.raises(ValueError):
            api.spec_tree_attention_shared(*good.values(), **kw)


def test_oracle_equals_the_one_without_sharing():
    rng = np.random.default_rng(0)
    B, N, Hq, Hkv, D = 3, 4, 4, 2, 8
    par = np.array([[-1, 0, 0, 2]] * B, dtype=np.int32)
    q = rng.normal(size=(B, N, Hq, D))
    kp, vp = (rng.normal(size=(2, Hkv, 9, D)) for _ in range(2))
    k, v = (rng.normal(size=(B, Hkv, 12, D)) for _ in range(2))
    pre, slen = [0, 5, 2], [7, 0]
    out, _, _, _ = oracle.tree_attention_shared(
        q, kp, vp, slen, [0, 2, 3], k, v, pre, tree_mask(par)[1], 0.4)
    for b in range(B):
        g = int(b == 2)
        cat = lambda x, y: np.concatenate([x[g:g + 1, :, :slen[g]],
                                           y[b:b + 1]], 2)
        want = tree_attention(q[b:b + 1], cat(kp, k), cat(vp, v),
                              [slen[g] + pre[b]], par[:1], 0.4)
        assert np.allclose(out[b], want[0])
