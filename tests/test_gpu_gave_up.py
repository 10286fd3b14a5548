"""Attention rows of a CTA one of whose bounded waits gave up come back as NaN,
in out and lse, and through the join of a split call; every other row is what
it was.  No wait is made to run out: a build of the two tensor-core kernels
with SV_TEST_GAVE_UP reads the flag of CTA 0 as set, after all of its waits.
"""

import os
import subprocess

import numpy as np
import pytest
import torch

from tests._parity import lib_ready
from tests.test_gpu_kv4 import _gen, _i32, _words, api, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def marked(tmp_path_factory):
    """The library with the flagged kernels, linked with the built objects."""
    lib_ready()
    from speculative_decoding_verification_tree_gb300 import _lib, build
    d = tmp_path_factory.mktemp("gave_up")
    names = ("kv4_attn_tc", "tree_attn")
    jobs = [subprocess.Popen(
        [build._nvcc(), *build.ARCH, *build.FLAGS, "-DSV_TEST_GAVE_UP", "-c",
         os.path.join(build.CSRC, n + ".cu"), "-o", str(d / (n + ".o"))])
        for n in names]
    assert [j.wait() for j in jobs] == [0, 0]
    objs = [str(d / (n + ".o")) for n in names]
    rest = {os.path.basename(s)[:-3] for s in build._inputs()[0]} - set(names)
    objs += [os.path.join(build.BUILD, n + ".o") for n in sorted(rest)]
    so = str(d / "libspecverify_gave_up.so")
    subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-o", so, *objs],
                   check=True)
    kept = _lib._lib
    _lib._lib = None
    lib = _lib.load(so)
    _lib._lib = kept
    return lib


def both(monkeypatch, marked, call):
    """The call's results from the library and from the marked build."""
    from speculative_decoding_verification_tree_gb300 import _lib
    base = call()
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(_lib, "_lib", marked)
        got = call()
        torch.cuda.synchronize()
    return base, got


def check(base, got, rows):
    """rows [B, N, Hq]: those of CTA 0."""
    (o0, l0), (o1, l1) = base, got
    assert torch.isfinite(o0.float()).all() and torch.isfinite(l0).all()
    assert torch.isnan(o1[rows].float()).all() and torch.isnan(l1[rows]).all()
    assert torch.equal(o1[~rows], o0[~rows])
    assert torch.equal(l1[~rows], l0[~rows])


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("N,Hq,Hkv,S,tile", [
    (20, 8, 2, 200, 128),       # one tile, unsplit
    (60, 8, 1, 200, 256),       # 480 rows: two CTAs of two tiles
    (20, 8, 2, 6000, 128),      # shares joined
    (60, 8, 1, 6000, 256),
])
def test_kv4_tree_rows_are_nan(monkeypatch, marked, N, Hq, Hkv, S, tile, D):
    B = 2
    prefix = [S // 3, S - N]    # CTA 0 takes the longer sequence
    cache, _ = make_cache(N, B, Hkv, S, D)
    q = torch.randn(B, N, Hq, D, generator=_gen(N), device="cuda").bfloat16()
    words = _words([[(1 << (i + 1)) - 1 for i in range(N)]] * B)
    call = lambda: api().spec_tree_attention_kv4(q, cache, _i32(prefix), words,
                                                 v_unit=0.125, lse=True)
    G = Hq // Hkv
    rows = np.zeros((B, N, Hq), dtype=bool)
    for r in range(min(tile, N * G)):
        rows[1, r // G, r % G] = True
    check(*both(monkeypatch, marked, call), torch.from_numpy(rows).cuda())


def test_bf16_tree_rows_are_nan(monkeypatch, marked):
    B, N, Hq, Hkv, D, S = 2, 20, 8, 2, 128, 300
    g = _gen(4)
    q, k, v = (torch.randn(*s, D, generator=g, device="cuda").bfloat16()
               for s in ((B, N, Hq), (B, Hkv, S), (B, Hkv, S)))
    words = _words([[(1 << (i + 1)) - 1 for i in range(N)]] * B)
    prefix = [S - N, 40]
    call = lambda: api().spec_tree_attention_lse(q, k, v, _i32(prefix), words)
    base, got = both(monkeypatch, marked, call)
    rows = torch.zeros(B, N, Hq, dtype=torch.bool, device="cuda")
    rows[0, :, :Hq // Hkv] = True
    check(base, got, rows)
