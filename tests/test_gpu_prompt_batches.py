"""Batches on both sides of the number of prompts up to which units are taken in
order of length, one long prompt at either end; tolerances of test_gpu_prompt.py.
"""

import numpy as np
import pytest

from tests._parity import lib_ready
from tests.test_gpu_prompt import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.mark.parametrize("B", [31, 32, 33, 47, 48, 49, 64, 65])
@pytest.mark.parametrize("D", [128, 64])
def test_batches(B, D):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 150, size=B).tolist()
    run(lens, 8, 2, D, seed=B)
    lens = rng.integers(1, 40, size=B)
    lens[-1] = 700
    run(lens.tolist(), 4, 2, D, seed=B + 1)
    run(lens[::-1].tolist(), 2, 1, D, seed=B + 2)
