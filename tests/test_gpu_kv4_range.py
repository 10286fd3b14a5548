"""Query rows, units and scales at the ends of what the 4-bit attention and
the weights accept: the factor scale log2(e) unit 2^e of a row (e the exponent
of its largest element) leaves float32's range long before the scores do.
Scores far below 2^-24 give the plain mean of what a row sees; the bounds are
test_gpu_kv4.py's.
"""

import math

import numpy as np
import pytest
import torch

from tests._parity import lib_ready
from tests.test_gpu_kv4 import (_gen, _i32, _words, api, check_attention,
                                make_cache)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("N,Hq", [(1, 1), (3, 4), (5, 4), (8, 4), (10, 4),
                                  (60, 4)])      # 1 to 240 rows a head
@pytest.mark.parametrize("unit,scale,mag", [
    (2.0 ** -64, 0.088, 1e-30),
    (1.0, 1e-38, 1e-9),
    (2.0 ** -64, 1e-38, 1e-37),
    (2.0 ** 64, 1e30, 0.0),
    (2.0 ** 64, 3.3e38, 0.0),
])
def test_row_factors_outside_float32(unit, scale, mag, N, Hq, D):
    prefix = [150, 0, 3]           # masked keys in every last block
    B, S = len(prefix), max(prefix) + N + 5
    cache, vals = make_cache(N, B, 1, S, D, k_unit=unit)
    q = (torch.randn(B, N, Hq, D, generator=_gen(N), device="cuda") * mag
         ).bfloat16()
    words = [[(1 << (i + 1)) - 1 for i in range(N)]] * B
    out, lse = api().spec_tree_attention_kv4(
        q, cache, _i32(prefix), _words(words), scale=scale, k_unit=unit,
        v_unit=0.125, lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, q, vals, prefix, words, scale)
    # and the weights of the whole chain: 1 / (P + t + 1) a row and head.
    # lse errs by at most (100 log2(e) + 72) 2^-24 + ..., the exponential by
    # 2^-22, the sum of 240 terms by 2^-16: 2^-14 in all
    w = api().spec_kv_weights(q, cache, lse, _i32(prefix), _i32([N] * B),
                              scale=scale, k_unit=unit)
    torch.cuda.synchronize()
    for b, P in enumerate(prefix):
        want = np.zeros(P + N)
        for t in range(N):
            want[:P + t + 1] += Hq / (P + t + 1)
        got = w[b, 0, :P + N].double().cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -14 * want).all()


def test_factor_of_a_zero_row_over_a_bf16_cache():
    B, N, Hq, D, P = 1, 4, 4, 128, 90
    k = torch.randn(B, 1, P + N, D, generator=_gen(1), device="cuda").bfloat16()
    q = torch.zeros(B, N, Hq, D, device="cuda", dtype=torch.bfloat16)
    words = _words([[(1 << (i + 1)) - 1 for i in range(N)]])
    _, lse = api().spec_tree_attention_lse(q, k, k, _i32([P]), words,
                                           scale=3.3e38)
    w = api().spec_kv_weights(q, k, lse, _i32([P]), _i32([N]), scale=3.3e38)
    torch.cuda.synchronize()
    want = sum(Hq / (P + t + 1) for t in range(N))
    assert torch.allclose(lse[0, :, 0].cpu(), torch.tensor(
        [math.log2(P + t + 1) for t in range(N)]), rtol=0, atol=2.0 ** -15)
    assert np.allclose(w[0, 0, :P].cpu().numpy(), want, rtol=2.0 ** -14)


@pytest.mark.parametrize("kind", ["kv4", "bf16"])
def test_rows_that_saw_nothing_add_nothing_to_nan_keys(kind):
    """lse = -inf: nothing is added, also where a key is NaN or a score
    overflows; the other rows' weights reach every position they see."""
    B, N, Hq, D, P = 1, 9, 2, 128, 700
    g = _gen(5)
    q = torch.randn(B, N, Hq, D, generator=g, device="cuda").bfloat16()
    k = torch.randn(B, 1, P + N, D, generator=g, device="cuda").bfloat16()
    if kind == "kv4":
        cache = api().kv4_cache(B, 1, P + N, D)
        kk = k.transpose(1, 2).contiguous()
        api().spec_kv4_append(kk, kk, _i32([0]), cache)
        k = cache[:2]
    lse = torch.full((B, N, Hq), 9.0, device="cuda")
    w0 = torch.rand(B, 1, P + N, generator=g, device="cuda")
    lse[0, 1:] = float("-inf")
    args = (_i32([P]), _i32([N]))
    one = api().spec_kv_weights(q, k, lse, _i32([P]), _i32([1]), weights=w0)
    got = api().spec_kv_weights(q, k, lse, *args, weights=w0)
    torch.cuda.synchronize()
    assert torch.equal(got[:, :, :P + 1], one[:, :, :P + 1])
    assert (got[:, :, P + 1:] == 0).all()
    # now no row sees anything, and keys are NaN
    lse[:] = float("-inf")
    if kind == "kv4":
        cache.k_scale[0, 0, 5::7] = 0x7F
    else:
        k[0, 0, 5::7] = float("nan")
    got = api().spec_kv_weights(q, k, lse, *args, weights=w0)
    huge = api().spec_kv_weights(q, k, lse, *args, scale=3e38, weights=w0)
    torch.cuda.synchronize()
    for x in (got, huge):
        assert torch.equal(x[:, :, :P], w0[:, :, :P])
        assert (x[:, :, P:] == 0).all()
