"""Shared-prefix calls whose pieces are the last step of one unit and the first of
the next: units of an odd number of steps in pieces of two.  A tile then takes part
in neither unit, twice in a row.  Every call is right (tolerances of
test_gpu_shared.py) and repeats its bits.
"""

import pytest
import torch

from tests._parity import lib_ready
from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu

CASES = [  # shared lengths, group starts, own prefixes, N, Hq, Hkv
    ([220], [0, 1], [1], 1, 12, 3),
    ([129], [0, 1], [0], 1, 4, 2),
    ([256], [0, 2], [0, 5], 1, 8, 8),           # four steps a unit
    ([200], [0, 20], [3] * 20, 1, 8, 2),
    ([200] * 12, list(range(13)), [7] * 12, 1, 32, 8),
    ([500] * 7, list(range(8)), [7] * 7, 2, 32, 8),
    ([60] * 30, list(range(31)), [130] * 30, 1, 6, 3),
    ([200, 129, 0, 390], [0, 1, 2, 3, 4], [0, 100, 300, 6], 5, 16, 4),
    ([1], [0, 1], [200], 16, 64, 8),            # one tile of rows, all own
]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0][:2]}-{c[3:]}")
@pytest.mark.parametrize("D", [128, 64])
def test_short_pieces(case, D):
    c = Case(*case, D, seed=len(case[0]))
    first = c.run()
    c.check(*first)
    for _ in range(100):
        assert all(torch.equal(x, y) for x, y in zip(first, c.run()))
