"""Attention over packed prompts on the GPU vs the oracle.

Tolerance, element by element, with A = sum_s w_s |v_s| (the softmax-weighted
magnitudes) and n the keys of a prompt:

* the output's rounding to bf16: 2^-8 |o|, and the weights' rounding to bf16 for
  the second product: 2^-8 A;
* a score is a float32 sum of D products of bf16 values (exact), scaled by one
  FMA: e = 2^-17 max_s scale sum_d |q_d k_d| covers D additions at 2^-24 each.
  It shifts every weight by a factor e^(+-e), numerator and denominator: 2 e A;
* float32 accumulation over n keys, 16 at a time in the products and eight
  partial sums joined, and the hardware exponential's 2^-22:
  (n / 16 + 64) 2^-23 A.

The normaliser (base 2): log2(e) e for the scores, the sum's relative error
(n / 4 + 64) 2^-24 log2(e), and 2^-21 |lse| for its own float32 steps.
"""

import numpy as np
import pytest
import torch

from oracle import prompt as oracle
from tests._parity import lib_ready, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def api():
    from speculative_decoding_verification_tree_gb300 import api as a
    return a


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(T, Hq, Hkv, D, seed=0, std=1.0, fused=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda")
         * std).bfloat16()
    parts = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    return parts if fused else tuple(t.contiguous() for t in parts)


def bounds(o, lse, mag, sm, n):
    """Tolerances of outputs and normalisers."""
    e = 2.0 ** -17 * sm
    tol = (2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * e[..., None]
           + (n / 16 + 64) * 2.0 ** -23) * mag + 1e-30)
    tl = 1.4427 * (e + (n / 4 + 64) * 2.0 ** -24) + 2.0 ** -21 * np.abs(lse)
    return tol, tl


def check(q, k, v, lens, out, lse, scale, first=0):
    starts = [first]
    for n in lens:
        starts.append(starts[-1] + n)
    o, l, mag, sm = oracle.prompt_attention(np64(q), np64(k), np64(v), starts,
                                            scale)
    tol, tl = bounds(o, l, mag, sm, max(lens))
    live = ~np.isnan(l)
    err = np.abs(np64(out) - o)
    assert (err <= tol)[live].all(), float((err / tol)[live].max())
    assert (np.abs(np64(lse) - l) <= tl)[live].all()


def run(lens, Hq, Hkv, D, seed=0, std=1.0, fused=False, scale=None):
    T = sum(lens)
    q, k, v = make(T, Hq, Hkv, D, seed, std, fused)
    starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    out, lse = api().spec_prompt_attention(q, k, v, i32(starts), lse=True,
                                           scale=scale)
    check(q, k, v, lens, out, lse, scale or D ** -0.5)
    return q, k, v, starts, out, lse


LENS = [[1], [1, 1, 1], [2], [63, 64, 65], [127, 128, 129, 1], [255, 256, 257],
        [0, 5, 0, 300, 0], [700], [33, 900, 1, 410]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("D", [128, 64])
def test_lengths(lens, D):
    run(lens, 8, 2, D, seed=len(lens))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (2, 1), (14, 2), (10, 2),
                                    (32, 8), (48, 3), (71, 1), (128, 1),
                                    (65, 1)])
@pytest.mark.parametrize("D", [128, 64])
def test_head_layouts(Hq, Hkv, D):
    run([130, 1, 301], Hq, Hkv, D, seed=Hq, fused=True)


def test_long_prompts():
    run([2500], 1, 1, 128, seed=1)
    run([2049, 1000], 4, 1, 64, seed=2)


def test_many_prompts():
    """More prompts than are ordered by length, most of them short."""
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 60, size=700).tolist()
    lens[333] = 1500
    run(lens, 4, 2, 128, seed=3)
    run([1] * 400, 8, 2, 64, seed=4)
    run(rng.integers(0, 90, size=256).tolist(), 8, 4, 64, seed=5)


@pytest.mark.parametrize("D", [128, 64])
def test_moving_maxima(D):
    """Scores whose maximum keeps growing towards either end, far past the
    distance at which a row's reference moves."""
    T = 600
    q, k, v = make(T, 2, 1, D, seed=6)
    for sign in (1, -1):
        ramp = torch.linspace(-1, 1, T, device="cuda")[:, None, None] * sign
        k2 = (k.float() * 0.1 + ramp * 4).bfloat16()
        q2 = (q.float() * 0.1 + 2).bfloat16()
        out, lse = api().spec_prompt_attention(q2, k2, v, i32([0, T]), lse=True,
                                               scale=1.0)
        check(q2, k2, v, [T], out, lse, 1.0)


def test_tokens_outside_every_prompt_stay():
    q, k, v = make(500, 8, 2, 128, seed=7)
    out = torch.full((500, 8, 128), 7.0, device="cuda").bfloat16()
    lse = torch.full((500, 8), 7.0, device="cuda")
    r = api().spec_prompt_attention(q, k, v, i32([40, 170, 170, 333]), out=out,
                                    lse=lse)
    assert r[0] is out and r[1] is lse
    check(q, k, v, [130, 0, 163], out, lse, 128 ** -0.5, first=40)
    for t in (out, lse):
        assert (t[:40] == 7).all() and (t[333:] == 7).all()
    # bounds outside the tensor are clamped, a descending pair is empty: prompts
    # 0..99, none, 50..59 and 60..499, which leaves tokens 50..99 to several
    api().spec_prompt_attention(q, k, v, i32([-5, 100, 50, 60, 900]), out=out,
                                lse=lse)
    check(q[:50], k[:50], v[:50], [50], out[:50], lse[:50], 128 ** -0.5)
    o, l, mag, sm = oracle.prompt_attention(np64(q), np64(k), np64(v),
                                            [60, 500], 128 ** -0.5)
    tol, tl = bounds(o, l, mag, sm, 440)
    assert (np.abs(np64(out) - o) <= tol)[100:].all()
    assert (np.abs(np64(lse) - l) <= tl)[100:].all()


@pytest.mark.parametrize("D", [128, 64])
def test_nan_and_infinity_reach_later_tokens_only(D):
    lens = [300, 200]
    q, k, v = make(500, 8, 2, D, seed=8)
    start = i32([0, 300, 500])
    base, lse0 = api().spec_prompt_attention(q, k, v, start, lse=True)
    for pos in (0, 70, 128, 255, 299, 300, 430):
        end = 300 if pos < 300 else 500
        for val in (float("nan"), float("inf"), -float("inf")):
            v2 = v.clone()
            v2[pos, 1, 5] = val
            out, lse = api().spec_prompt_attention(q, k, v2, start, lse=True)
            want = base.clone()
            want[pos:end, 4:, 5] = val
            assert torch.equal(lse, lse0)
            assert torch.equal(torch.nan_to_num(out, 77., 88., 99.),
                               torch.nan_to_num(want, 77., 88., 99.))
        k2 = k.clone()
        k2[pos, 0, 3] = float("nan")
        out, lse = api().spec_prompt_attention(q, k2, v, start, lse=True)
        assert torch.isnan(out[pos:end, :4]).all()
        assert torch.isnan(lse[pos:end, :4]).all()
        keep = torch.ones(500, 8, dtype=torch.bool, device="cuda")
        keep[pos:end, :4] = False
        assert torch.equal(out[keep], base[keep])
        assert torch.equal(lse[keep], lse0[keep])
    # both infinities in one column meet as NaN
    v2 = v.clone()
    v2[10, 0, 0], v2[20, 0, 0] = float("inf"), -float("inf")
    out, _ = api().spec_prompt_attention(q, k, v2, start)
    assert (out[10:20, :4, 0] == float("inf")).all()
    assert torch.isnan(out[20:300, :4, 0]).all()
    assert torch.isfinite(out[300:]).all()


@pytest.mark.parametrize("D", [128, 64])
def test_many_nan_values_over_many_units(D):
    """Scattered NaN values in prompts of many units: each reaches its own and
    later tokens of its prompt, in its head's column, while CTAs go on to their
    next units."""
    lens, Hkv = [3000, 1, 700, 2500, 64], 8
    T = sum(lens)
    q, k, v = make(T, 16, Hkv, D, seed=12)
    rng = np.random.default_rng(12)
    at = (rng.integers(0, T, 400), rng.integers(0, Hkv, 400),
          rng.integers(0, D, 400))
    at = tuple(torch.from_numpy(x).cuda() for x in at)
    starts = np.concatenate([[0], np.cumsum(lens)])
    v[at] = 0
    base, lse0 = api().spec_prompt_attention(q, k, v, i32(starts), lse=True)
    v[at] = float("nan")
    out, lse = api().spec_prompt_attention(q, k, v, i32(starts), lse=True)
    assert torch.equal(lse, lse0)
    hit = torch.isnan(v)                            # [T, Hkv, D]
    for a, z in zip(starts, starts[1:]):
        hit[a:z] = hit[a:z].cumsum(0) > 0
    hit = hit.repeat_interleave(2, 1)
    assert torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], base[~hit])


def test_rows_past_2_31_elements():
    """600 K tokens of 32 heads: q and out pass 2^31 elements."""
    n, L = 2350, 257
    T = n * L
    q = torch.empty(T, 32, 128, dtype=torch.bfloat16, device="cuda")
    q.normal_()
    k = torch.randn(T, 1, 128, device="cuda").bfloat16()
    v = torch.randn(T, 1, 128, device="cuda").bfloat16()
    start = torch.arange(n + 1, device="cuda", dtype=torch.int32) * L
    out, lse = api().spec_prompt_attention(q, k, v, start, lse=True)
    for b in (0, n - 1):
        r = slice(b * L, b * L + L)
        check(q[r], k[r], v[r], [L], out[r], lse[r], 128 ** -0.5)


def test_streams_and_graphs():
    q, k, v = make(900, 8, 2, 128, seed=9)
    start = i32([0, 400, 900])
    call = lambda: api().spec_prompt_attention(q, k, v, start, lse=True)
    base = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = api().spec_prompt_attention(q, k, v, start, lse=True, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(base, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    q.copy_(make(900, 8, 2, 128, seed=10)[0])
    start.copy_(i32([0, 123, 890]))
    g.replay()
    want = call()
    assert torch.equal(out[0][:890], want[0][:890])
    assert torch.equal(out[1][:890], want[1][:890])
    check(q, k, v, [123, 767], out[0], out[1], 128 ** -0.5)
