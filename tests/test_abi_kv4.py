"""Refusals of the 4-bit cache, weight and eviction entry points: C ABI
argument errors (no device work) and the wrappers' checks (no library call)."""

import ctypes

import pytest
import torch

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


@pytest.mark.parametrize("name", ["spec_kv4_append", "spec_kv4_read"])
def test_append_and_read_argument_errors(lib, name):
    def call(a=FAKE, b=FAKE, c=FAKE, d=FAKE, e=FAKE, x=FAKE, y=FAKE, B=2, n=3,
             Hkv=2, D=128, S=16, ku=1.0, vu=0.5):
        if name == "spec_kv4_append":   # k, v, prefix; then the cache
            return lib.raw(name, x, y, e, B, n, Hkv, D, S, ku, vu, a, b, c, d,
                           None)
        return lib.raw(name, a, b, c, d, e, B, n, Hkv, D, S, ku, vu, x, y, None)
    assert call(B=-1) == lib.SPEC_ERR_SHAPE
    assert call(n=-1) == lib.SPEC_ERR_SHAPE
    assert call(Hkv=0) == lib.SPEC_ERR_SHAPE
    assert call(S=-1) == lib.SPEC_ERR_SHAPE
    assert call(B=65535, n=1 << 30, Hkv=64) == lib.SPEC_ERR_SHAPE
    for D in (0, 32, 96, 256):
        assert call(D=D) == lib.SPEC_ERR_UNSUPPORTED
    for u in (0.0, -1.0, 0.3, 3.0, 2.0 ** -65, 2.0 ** 65, float("nan"),
              float("inf")):
        assert call(ku=u) == lib.SPEC_ERR_ARG
        assert call(vu=u) == lib.SPEC_ERR_ARG
    for kw in ({"a": None}, {"b": None}, {"c": None}, {"d": None}, {"e": None},
               {"x": None}, {"y": None}, {"a": ODD}, {"c": ODD}, {"x": ODD},
               {"y": ODD}, {"b": ODD4}, {"d": ODD4}, {"e": ODD2}):
        assert call(**kw) == lib.SPEC_ERR_ARG, kw
    assert call(B=0, a=None, x=None) == lib.SPEC_OK
    assert call(n=0, a=None, x=None) == lib.SPEC_OK


def test_attention_argument_errors(lib):
    # one long sequence leaves partial results; short ones need no workspace
    f = lib.raw("spec_tree_attention_kv4_workspace_bytes", 1, 1, 8, 2, 128,
                1 << 18)
    assert f > 0 and f % 256 == 0
    assert lib.raw("spec_tree_attention_kv4_workspace_bytes", 2, 8, 8, 2, 128,
                   64) == 0
    for bad in ((-1, 8, 8, 2, 128, 64), (2, 0, 8, 2, 128, 64),
                (2, 65, 8, 2, 128, 64), (2, 8, 7, 2, 128, 64),
                (2, 8, 8, 2, 96, 64), (2, 8, 8, 2, 128, 7)):
        assert lib.raw("spec_tree_attention_kv4_workspace_bytes", *bad) == 0

    def call(q=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pre=FAKE, mb=FAKE,
             B=2, N=8, Hq=8, Hkv=2, D=128, S=64, scale=0.1, ku=1.0, vu=1.0,
             out=FAKE, lse=None, ws=FAKE, nbytes=f):
        return lib.raw("spec_tree_attention_kv4", q, kc, ks, vc, vs, pre, mb,
                       B, N, Hq, Hkv, D, S, scale, ku, vu, out, lse, ws,
                       nbytes, None)
    for kw in (dict(B=-1), dict(B=65536), dict(N=0), dict(N=65), dict(Hq=7),
               dict(Hkv=0), dict(S=7), dict(S=(1 << 30) + 1),
               dict(Hq=1 << 30, Hkv=1), dict(B=65535, Hq=1 << 30, Hkv=1 << 30)):
        assert call(**kw) == lib.SPEC_ERR_SHAPE, kw
    assert call(D=32) == lib.SPEC_ERR_UNSUPPORTED
    for kw in (dict(scale=0.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(ku=3.0), dict(vu=0.0),
               dict(q=None), dict(kc=None), dict(ks=None), dict(vc=None),
               dict(vs=None), dict(pre=None), dict(mb=None), dict(out=None),
               dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD),
               dict(ks=ODD4), dict(vs=ODD4), dict(mb=ODD4), dict(pre=ODD2),
               dict(lse=ODD2)):
        assert call(**kw) == lib.SPEC_ERR_ARG, kw
    long = dict(B=1, N=1, S=1 << 18)
    for kw in (dict(ws=None), dict(ws=ODD), dict(nbytes=f - 256)):
        assert call(**long, **kw) == lib.SPEC_ERR_WORKSPACE, kw
    assert call(B=0, q=None, ws=None, nbytes=0) == lib.SPEC_OK


def test_attention_lse_argument_errors(lib):
    def call(B=2, N=8, D=128, q=FAKE, lse=FAKE, scale=0.1):
        return lib.raw("spec_tree_attention_lse", q, FAKE, FAKE, FAKE, FAKE, B,
                       N, 8, 2, D, 64, scale, FAKE, lse, None)
    assert call(lse=None) == lib.SPEC_ERR_ARG
    assert call(lse=ODD2) == lib.SPEC_ERR_ARG
    assert call(q=None) == lib.SPEC_ERR_ARG
    assert call(scale=0.0) == lib.SPEC_ERR_ARG
    assert call(N=65) == lib.SPEC_ERR_SHAPE
    assert call(D=64) == lib.SPEC_ERR_UNSUPPORTED
    assert call(B=0, q=None, lse=None) == lib.SPEC_OK


def test_weights_argument_errors(lib):
    def call(q=FAKE, k=FAKE, ks=FAKE, lse=FAKE, pre=FAKE, n=FAKE, nodes=FAKE,
             B=2, N=8, Hq=8, Hkv=2, D=128, S=64, scale=0.1, ku=1.0, w=FAKE,
             out=FAKE):
        return lib.raw("spec_kv_weights", q, k, ks, lse, pre, n, nodes, B, N,
                       Hq, Hkv, D, S, scale, ku, w, out, None)
    for kw in (dict(B=-1), dict(B=65536), dict(Hq=1 << 30, Hkv=1),
               dict(S=(1 << 30) + 1), dict(N=0), dict(N=65), dict(Hq=7), dict(S=7)):
        assert call(**kw) == lib.SPEC_ERR_SHAPE, kw
    assert call(D=80) == lib.SPEC_ERR_UNSUPPORTED
    for kw in (dict(scale=-1.0), dict(ku=1.5), dict(ks=None, ku=2.0),
               dict(q=None), dict(k=None), dict(lse=None), dict(pre=None),
               dict(n=None), dict(out=None), dict(q=ODD), dict(k=ODD),
               dict(ks=ODD4), dict(lse=ODD2), dict(w=ODD2), dict(out=ODD2),
               dict(nodes=ODD2), dict(n=ODD2), dict(pre=ODD2)):
        assert call(**kw) == lib.SPEC_ERR_ARG, kw
    assert call(B=0, q=None, out=None) == lib.SPEC_OK


def test_evict_argument_errors(lib):
    def call(w=FAKE, n=FAKE, B=2, Hkv=2, S=64, budget=16, recent=4,
             planes=(FAKE.value,), outs=(FAKE.value + 4096,), rows=(64,),
             S_out=32, wo=None, kept=FAKE, new=FAKE, n_planes=None,
             arrays=True):
        k = len(planes)
        P = (ctypes.c_void_p * max(k, 1))(*planes) if arrays else None
        O = (ctypes.c_void_p * max(k, 1))(*outs) if arrays else None
        R = (ctypes.c_int * max(k, 1))(*rows) if arrays else None
        return lib.raw("spec_kv_evict", w, n, B, Hkv, S, budget, recent,
                       k if n_planes is None else n_planes, P, O, R, S_out, wo,
                       kept, new, None)
    for kw in (dict(B=-1), dict(Hkv=0), dict(S=-1), dict(S_out=-1),
               dict(budget=0), dict(budget=33), dict(recent=-1),
               dict(recent=17), dict(n_planes=-1), dict(n_planes=9),
               dict(rows=(0,)), dict(rows=(65537,)),
               dict(B=65536, Hkv=65536), dict(S=(1 << 30) + 1),
               dict(S_out=(1 << 30) + 1)):
        assert call(**kw) == lib.SPEC_ERR_SHAPE, kw
    for kw in (dict(n=ODD4, new=ODD4),                 # lengths in place
               dict(w=None), dict(n=None), dict(kept=None), dict(new=None),
               dict(planes=(None,)), dict(outs=(None,)), dict(arrays=False),
               dict(w=ODD2), dict(n=ODD2), dict(kept=ODD2), dict(new=ODD2),
               dict(wo=ODD2), dict(wo=FAKE),           # in place, S_out != S
               dict(outs=(FAKE.value,))):
        assert call(**kw) == lib.SPEC_ERR_ARG, kw
    assert call(B=0, w=None, planes=(None,), outs=(None,)) == lib.SPEC_OK


def test_evict_refuses_arrays_that_overlap(lib):
    """2 x 2 pairs of 64 positions; every array apart but for the ones named.
    All calls are refused before any device work."""
    at = lambda i: FAKE.value + (i << 20)
    W, N, K, V, KO, VO, WO, KEPT, NEW = map(at, range(9))

    def call(planes=(K, V), outs=(K, V), rows=(64, 64), w=W, wo=W, n=N,
             kept=KEPT, new=NEW, S=64, S_out=64):
        k = len(planes)
        return lib.raw("spec_kv_evict", w, n, 2, 2, S, 16, 4, k,
                       (ctypes.c_void_p * k)(*planes),
                       (ctypes.c_void_p * k)(*outs), (ctypes.c_int * k)(*rows),
                       S_out, wo, kept, new, None)
    size = 2 * 2 * 64 * 64
    for kw in (dict(planes=(K, K), outs=(K, K)),          # twice in place
               dict(planes=(K, V), outs=(KO, KO)),        # one output for two
               dict(planes=(K, V), outs=(V, K)),          # exchanged
               dict(planes=(K, V), outs=(KO, K)),         # over another's input
               dict(outs=(K + 64, VO)),                   # shifted by a row
               dict(outs=(KO, KO + size - 4)),            # their last word
               dict(planes=(K, W), outs=(K, W), rows=(64, 4)),   # moved twice
               dict(planes=(K, W), outs=(K, VO), rows=(64, 4)),  # moves first
               dict(planes=(K, V), outs=(W, V), wo=None),
               dict(wo=K, outs=(KO, VO)), dict(wo=KO, outs=(KO, VO)),
               dict(wo=W + 4), dict(new=N), dict(new=N + 4), dict(kept=N),
               dict(kept=W), dict(kept=K + size - 4), dict(kept=WO, wo=WO),
               dict(new=W), dict(new=V), dict(new=KEPT), dict(wo=N, outs=(KO, VO)),
               dict(outs=(N, VO))):
        assert call(**kw) == lib.SPEC_ERR_ARG, kw


def test_wrappers_reject_malformed_tensors():
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    B, N, Hq, Hkv, D, S = 2, 3, 4, 2, 128, 16
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    cache = api.KV4Cache(z(B, Hkv, S, 64, dt=u8), z(B, Hkv, S, 8, dt=u8),
                         z(B, Hkv, S, 64, dt=u8), z(B, Hkv, S, 8, dt=u8))
    k = z(B, N, Hkv, D, dt=bf)
    pre, q = z(B, dt=i32), z(B, N, Hq, D, dt=bf)
    mb = z(B, N, dt=torch.int64)
    with pytest.raises(ValueError):
        api.spec_kv4_append(k.float(), k, pre, cache)
    with pytest.raises(ValueError):
        api.spec_kv4_append(k, k[:, :2], pre, cache)
    with pytest.raises(ValueError):
        api.spec_kv4_append(k, k, pre.long(), cache)
    with pytest.raises(ValueError):  # three arrays are not a cache
        api.spec_kv4_append(k, k, pre, cache[:3])
    with pytest.raises(ValueError):  # scales of another head dim
        api.spec_kv4_read(cache._replace(v_scale=z(B, Hkv, S, 4, dt=u8)), pre, 2)
    with pytest.raises(ValueError):
        api.spec_tree_attention_kv4(q, cache, pre, mb.int())
    with pytest.raises(ValueError):
        api.spec_tree_attention_kv4(q[..., :64], cache, pre, mb)
    with pytest.raises(ValueError):  # CPU tensors reach no kernel
        api.spec_kv4_append(k, k, pre, cache)
    lse = z(B, N, Hq)
    with pytest.raises(ValueError):
        api.spec_kv_weights(q, cache.k, lse, pre, pre)    # codes alone
    with pytest.raises(ValueError):
        api.spec_kv_weights(q, cache, lse.double(), pre, pre)
    with pytest.raises(ValueError):
        api.spec_kv_weights(q, cache, lse, pre, pre, z(B, N + 1, dt=i32))
    w = z(B, Hkv, S)
    with pytest.raises(ValueError):
        api.spec_kv_evict(w, pre, cache, budget=0, recent=0)
    with pytest.raises(ValueError):   # planes do not pair up
        api.spec_kv_evict(w, pre, cache, budget=4, recent=0,
                          planes_out=cache[:2])
    with pytest.raises(ValueError):   # another dtype
        api.spec_kv_evict(w, pre, cache[:1], budget=4, recent=0,
                          planes_out=(z(B, Hkv, 4, 64),))
    with pytest.raises(ValueError):   # in place moves the weights too
        api.spec_kv_evict(w, pre, cache, budget=4, recent=0,
                          weights_out=w.clone())
    with pytest.raises(ValueError):
        api.spec_kv_evict(w, pre, (cache.k,) * 9, budget=4, recent=0)


def test_wrappers_match_their_signatures(monkeypatch):
    calls = []

    def fake(name, *args):
        types = _lib._SIGNATURES[name][1]
        assert len(args) == len(types), name
        for a, t in zip(args, types):
            if a is not None and t in (ctypes.c_int, ctypes.c_float):
                t(a)
        calls.append(name)
        return 256
    monkeypatch.setattr(_lib, "call", fake)
    monkeypatch.setattr(api, "_index", lambda t: 0)
    monkeypatch.setattr(api, "_arg", lambda *a: FAKE.value)
    monkeypatch.setattr(api, "_raw_stream", lambda i: 0)
    monkeypatch.setattr(api, "_current_device", lambda: 0)
    monkeypatch.setattr(api, "_alloc", lambda shape, dtype, dev, stream,
                        make=torch.empty: make(shape, dtype=dtype))
    B, N, Hq, Hkv, D, S = 2, 3, 4, 2, 64, 16
    cache = api.kv4_cache(B, Hkv, S, D, device="cpu")
    k = torch.zeros(B, N, Hkv, D, dtype=torch.bfloat16)
    q = torch.zeros(B, N, Hq, D, dtype=torch.bfloat16)
    i = torch.zeros(B, dtype=torch.int32)
    assert api.spec_kv4_append(k, k, i, cache) is cache
    rk, rv = api.spec_kv4_read(cache, i, N)
    assert rk.shape == rv.shape == k.shape
    out, lse = api.spec_tree_attention_kv4(
        q, cache, i, torch.zeros(B, N, dtype=torch.int64), lse=True)
    assert out.shape == q.shape and lse.shape == (B, N, Hq)
    w = api.spec_kv_weights(q, cache, lse, i, i)
    assert w.shape == (B, Hkv, S)
    kept, n = api.spec_kv_evict(w, i, cache, budget=5, recent=2)
    assert kept.shape == (B, Hkv, 5) and n.shape == (B,)
    bits = torch.zeros(B, N, dtype=torch.int64)
    bf = torch.zeros(B, Hkv, S, D, dtype=torch.bfloat16)
    out, lse = api.spec_tree_attention_lse(q, bf, bf, i, bits)
    assert out.shape == q.shape and lse.shape == (B, N, Hq)
    assert calls == ["spec_kv4_append", "spec_kv4_read",
                     "spec_tree_attention_kv4_workspace_bytes",
                     "spec_tree_attention_kv4", "spec_kv_weights",
                     "spec_kv_evict", "spec_tree_attention_lse"]
