"""Lengths outside their range in shared-prefix attention count as the nearest one
inside, outputs and normalisers compared with the oracle at that length
(tolerances of test_gpu_shared.py).
"""

import pytest
import torch

from tests._parity import lib_ready
from tests.test_gpu_shared import Case, api, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("low", [-1, -3, -(1 << 31)])
def test_own_lengths_below_zero(low, D):
    """The drafted nodes then lie at positions 0 to N - 1."""
    c = Case([90], [0, 3], [0, 7, 20], 5, 8, 2, D, seed=6)
    c.k[0, :, 5:8] = 3.0        # what follows them is not seen
    c.v[0, :, 5:8] = 9.0
    a = list(c.args())
    a[7] = i32([low, 7, 20])
    c.check(*api().spec_tree_attention_shared(*a, scale=c.scale, lse=True))


@pytest.mark.parametrize("D", [128, 64])
def test_own_and_shared_lengths_past_the_end(D):
    c = Case([90, 33], [0, 2, 3], [40, 7, 40], 5, 8, 2, D, seed=7, slack=0)
    c.slen = [90, 90]           # the second prefix to its last position
    c.kp[1, :, 33:], c.vp[1, :, 33:] = 0.5, -0.25
    a = list(c.args())
    a[3] = i32([(1 << 31) - 1, 91])
    a[7] = i32([41, 7, (1 << 31) - 1])
    c.check(*api().spec_tree_attention_shared(*a, scale=c.scale, lse=True))


@pytest.mark.parametrize("D", [128, 64])
def test_shared_lengths_below_zero(D):
    c = Case([70, 30], [0, 1, 2], [9, 200], 3, 4, 1, D, seed=8)
    a = list(c.args())
    a[3] = i32([-5, 30])
    c.slen = [0, 30]
    out, lse = api().spec_tree_attention_shared(*a, scale=c.scale, lse=True)
    c.check(out, lse)
    assert torch.isfinite(out).all()
