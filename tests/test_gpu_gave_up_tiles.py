"""Rows of a CTA one of whose bounded waits gave up come back as NaN from the
prompt and shared-prefix attention, in out and lse, and through the join of a
cut unit; every other row is what it was.  No wait is made to run out: a build
with SV_TEST_GAVE_UP reads the flag of CTA 0 as set, after all of its waits.
"""

import os
import subprocess

import pytest
import torch

from tests._parity import lib_ready
from tests.test_gpu_gave_up import both, check
from tests.test_gpu_prompt import api, i32, make
from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def marked(tmp_path_factory):
    """The library with the flagged kernels, linked with the built objects."""
    lib_ready()
    from speculative_decoding_verification_tree_gb300 import _lib, build
    d = tmp_path_factory.mktemp("gave_up_tiles")
    names = ("prompt_attn", "shared_attn")
    jobs = [subprocess.Popen(
        [build._nvcc(), *build.ARCH, *build.FLAGS, "-DSV_TEST_GAVE_UP", "-c",
         os.path.join(build.CSRC, n + ".cu"), "-o", str(d / (n + ".o"))])
        for n in names]
    assert [j.wait() for j in jobs] == [0, 0]
    objs = [str(d / (n + ".o")) for n in names]
    rest = {os.path.basename(s)[:-3] for s in build._inputs()[0]} - set(names)
    objs += [os.path.join(build.BUILD, n + ".o") for n in sorted(rest)]
    so = str(d / "libspecverify_gave_up_tiles.so")
    subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-o", so, *objs],
                   check=True)
    kept = _lib._lib
    _lib._lib = None
    lib = _lib.load(so)
    _lib._lib = kept
    return lib


@pytest.mark.parametrize("D", [128, 64])
def test_prompt_rows_are_nan(monkeypatch, marked, D):
    """CTA 0 takes the longest unit: the last 64-position unit of the longest
    prompt, first key/value head (four query heads)."""
    q, k, v = make(420, 8, 2, D, seed=1)
    start = i32([0, 120, 420])
    call = lambda: api().spec_prompt_attention(q, k, v, start, lse=True)
    rows = torch.zeros(420, 8, dtype=torch.bool, device="cuda")
    rows[120 + 256:, :4] = True
    check(*both(monkeypatch, marked, call), rows)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("slen,N", [(0, 1), (9000, 1), (5000, 33)])
def test_shared_rows_are_nan(monkeypatch, marked, slen, N, D):
    """CTA 0 begins with the first unit: cut (long prefix), or with every other
    step of the call (two steps)."""
    c = Case([slen], [0, 1], [5], N, 8, 2, D, seed=2)
    rows = torch.zeros(1, N, 8, dtype=torch.bool, device="cuda")
    rows[:, :, :8 if slen == 0 else 4] = True
    base, got = both(monkeypatch, marked, c.run)
    if slen == 0:
        assert torch.isnan(got[0]).all() and torch.isnan(got[1]).all()
    else:
        check(base, got, rows)
