"""The last waits of the tile kernel's producer: for its last copy into every
stage of keys and values and into both query tiles.  A wait for a phase that does
not come would end after 2^31 cycles, about a second; calls of few and many
units, of one tile and two, an odd and an even number of each, stay far below it
(a tenth of a second allows for a busy host).
"""

import time

import pytest
import torch

from tests._parity import lib_ready
from tests.test_gpu_prompt import api, i32, make
from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def quick(call):
    call()
    torch.cuda.synchronize()
    best = 1.0
    for _ in range(3):
        t = time.perf_counter()
        call()
        torch.cuda.synchronize()
        best = min(best, time.perf_counter() - t)
    assert best < 0.1, best


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("lens", [
    [1], [64], [65], [128], [129], [300], [1] * 20, [40, 200], [65] * 39,
    [64] * 77 + [65] * 80, [5000], list(range(0, 900, 31))], ids=str)
def test_prompts_end_at_once(lens, D):
    T = sum(lens)
    q, k, v = make(T, 8, 2, D, seed=T)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    starts = i32(starts)
    quick(lambda: api().spec_prompt_attention(q, k, v, starts, lse=True))


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("case", [
    ([0], [0, 1], [0], 1, 8, 2), ([1], [0, 1], [0], 1, 8, 2),
    ([5000], [0, 2], [10, 900], 1, 32, 8),
    ([300], [0, 40], list(range(40)), 1, 8, 2),
    ([260, 511], [0, 1, 4], [33, 128, 0, 400], 60, 8, 2),
    ([260], [0, 2], [33, 140], 64, 32, 2),
    ([70] * 200, list(range(201)), [3] * 200, 1, 8, 2)],
    ids=lambda c: f"{c[0][:2]}-{c[3:]}")
def test_shared_calls_end_at_once(case, D):
    c = Case(*case, D, seed=3)
    a = c.args()
    quick(lambda: api().spec_tree_attention_shared(*a, scale=c.scale, lse=True))
