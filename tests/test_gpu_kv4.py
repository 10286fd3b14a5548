"""The 4-bit cache on the GPU vs the oracle: append, read, tree attention.

Append and read are exact.  Attention tolerance, element by element, with
A = sum_s w_s |v_s| (the softmax-weighted magnitudes, from the oracle):

* the output's rounding to bf16: 2^-8 |o|;
* the weights' rounding to fp16: 2^-11 A, and below the normal range 2^-25
  against weights lifted to at least 2^7 at the maximum: n 2^-32 max |v|;
* a score is a float32 sum of D products, scaled by one FMA: at most 2^-20 of
  scale sum_d |q_d k_d| (D <= 128 additions at 2^-24 each are 2^-17 at the
  very worst; the sum of magnitudes only bounds partial sums, so each step
  errs by 2^-24 of at most that sum and the fp16 operands are exact) -- taken
  as e = 2^-17 max_s scale sum_d |q_d k_d|, which also covers q's elements
  below 2^-14 of their row's largest.  It shifts every weight by a factor
  e^(+-e), numerator and denominator: 2 e A;
* float32 accumulation over n keys, 16 at a time in the products and eight
  partial sums joined: (n / 16 + 64) 2^-23 A.

The normaliser (base 2): log2(e) e for the scores, the sum's relative error
(n / 4 + 64) 2^-24 log2(e), and 2^-21 |lse| for its own float32 steps.
"""

import numpy as np
import pytest
import torch

import synth
from oracle import kv4
from oracle.tree import tree_mask
from tests._parity import lib_ready, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def api():
    from speculative_decoding_verification_tree_gb300 import api as a
    return a


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _words(bits):
    return torch.from_numpy(np.asarray(bits, dtype=np.uint64).view(np.int64)
                            ).cuda()


def random_parent(rng, B, N):
    return np.array([[-1 if j == 0 or rng.random() < 0.25 else
                      int(rng.integers(max(0, j - 6), j)) for j in range(N)]
                     for _ in range(B)], dtype=np.int32)


def make_cache(seed, B, Hkv, S, D, k_unit=1.0, v_unit=0.125, used=None):
    """A cache filled through the oracle's quantiser; positions at or behind
    used[b] hold bytes that stand for NaN."""
    a = api()
    rng = np.random.default_rng(seed)
    out = []
    for unit, std in ((k_unit, 1.0), (v_unit, 0.7)):
        x = torch.from_numpy(rng.normal(size=(B, Hkv, S, D)) * std
                             ).bfloat16().double().numpy()
        c, s = kv4.quantise(x, unit)
        if used is not None:
            for b in range(B):
                c[b, :, used[b]:] = 0xFF
                s[b, :, used[b]:] = 0x7F
        out += [c, s]
    cache = a.KV4Cache(*[torch.from_numpy(x).cuda() for x in out])
    vals = (kv4.values(out[0], out[1], k_unit),
            kv4.values(out[2], out[3], v_unit))
    return cache, vals


def attention_bounds(q, k, v, prefix, words, scale, lse):
    """Tolerances of out and lse, as derived above."""
    B, N, Hq, D = q.shape
    G = Hq // k.shape[1]
    ta = np.zeros((B, N, Hq, D))
    tl = np.zeros((B, N, Hq))
    for b in range(B):
        P = int(prefix[b])
        for i in range(N):
            word = int(words[b][i])
            keys = list(range(P)) + [P + j for j in range(N) if word >> j & 1]
            if not keys:
                continue
            n = P + N
            for h in range(Hq):
                kk, vv = k[b, h // G, keys], v[b, h // G, keys]
                s = scale * (kk @ q[b, i, h])
                w = np.exp(s - s.max())
                w /= w.sum()
                mag = scale * (np.abs(kk) @ np.abs(q[b, i, h])).max()
                e = mag * 2.0 ** -17
                A = w @ np.abs(vv)
                ta[b, i, h] = (2.0 ** -11 + 2 * e + (n / 16 + 64) * 2.0 ** -23
                               ) * A + n * 2.0 ** -32 * np.abs(vv).max()
                tl[b, i, h] = (np.log2(np.e) * (e + (n / 4 + 64) * 2.0 ** -24)
                               + 2.0 ** -21 * (abs(lse[b, i, h]) + 1))
    return ta, tl


def check_attention(out, lse, q, vals, prefix, words, scale):
    k, v = vals
    ref, rl = kv4.attention(np64(q), k, v, prefix, words, scale)
    ta, tl = attention_bounds(np64(q), k, v, prefix, words, scale,
                              np.where(np.isfinite(rl), rl, 0))
    got = np64(out)
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    worst = (err - (ta + 2.0 ** -8 * np.abs(ref))).max()
    assert worst <= 0, (worst, err.max())
    if lse is not None:
        gl = lse.double().cpu().numpy()
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(gl), empty)
        el = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl))
        assert (el <= tl).all(), (el - tl).max()


# ------------------------------------------------------------ append / read
@pytest.mark.parametrize("B,n,Hkv,D,S,unit", [
    (1, 1, 1, 64, 1, 1.0),
    (3, 5, 3, 128, 40, 0.125),
    (2, 60, 8, 128, 101, 4.0),
    (2, 33, 2, 64, 37, 2.0 ** -10),
])
def test_append_and_read_match_the_oracle(B, n, Hkv, D, S, unit):
    g = _gen(B * 100 + n)
    k = (torch.randn(B, n, Hkv, D, generator=g, device="cuda") * 3).bfloat16()
    v = (torch.randn(B, n, Hkv, D, generator=g, device="cuda") * 0.01).bfloat16()
    # exact borders: multiples of quarters of a power of two
    k[:, :, :, :16] = (torch.randint(-24, 25, (B, n, Hkv, 16), generator=g,
                                     device="cuda") / 4.0).bfloat16()
    pre = _i32([(7 * b) % max(1, S - n + 1) for b in range(B)])
    a = api()
    cache = a.kv4_cache(B, Hkv, S, D)
    for t in cache:
        t.fill_(0xA5)
    a.spec_kv4_append(k, v, pre, cache, k_unit=unit, v_unit=unit)
    rk, rv = a.spec_kv4_read(cache, pre, n, k_unit=unit, v_unit=unit)
    torch.cuda.synchronize()
    for x, (codes, scales), rd in ((k, cache[:2], rk), (v, cache[2:], rv)):
        wc, ws = kv4.quantise(np64(x), unit)
        want_c = np.full(codes.shape, 0xA5, dtype=np.uint8)
        want_s = np.full(scales.shape, 0xA5, dtype=np.uint8)
        for b in range(B):
            p = int(pre[b])
            want_c[b, :, p:p + n] = wc[b].transpose(1, 0, 2)
            want_s[b, :, p:p + n] = ws[b].transpose(1, 0, 2)
        assert np.array_equal(codes.cpu().numpy(), want_c)
        assert np.array_equal(scales.cpu().numpy(), want_s)
        assert np.array_equal(np64(rd), kv4.values(wc, ws, unit))


def test_append_every_bf16_magnitude():
    # every finite bf16 as a block's largest element, and against every
    # scale its neighbours choose: codes and scales equal the oracle's
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    x = bits.to(torch.int16).view(torch.bfloat16).cuda()
    n = (x.numel() + 7) // 8
    pad = torch.zeros(n * 8, dtype=torch.bfloat16, device="cuda")
    pad[:x.numel()] = x
    k = torch.zeros(1, n, 1, 128, dtype=torch.bfloat16, device="cuda")
    k[0, :, 0, ::16] = pad.view(n, 8)
    k[0, :, 0, 1::16] = -pad.view(n, 8) * 0.3125
    k[0, :, 0, 5::16] = pad.view(n, 8) * 0.5
    k[0, :, 0, 9::16] = pad.view(n, 8) * 0.1
    a = api()
    cache = a.kv4_cache(1, 1, n, 128)
    z = _i32([0])
    for unit in (1.0, 2.0 ** -20, 2.0 ** 33):
        a.spec_kv4_append(k, k, z, cache, k_unit=unit, v_unit=unit)
        torch.cuda.synchronize()
        c, s = kv4.quantise(np64(k), unit)
        for got, want in ((cache.k, c), (cache.v, c), (cache.k_scale, s)):
            assert np.array_equal(got.cpu().numpy()[0, 0], want[0, :, 0])


def test_append_special_values_and_positions_outside():
    a = api()
    k = torch.ones(3, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 1, 0, 17] = float("nan")
    k[0, 2, 0, 3] = float("-inf")
    cache = a.kv4_cache(3, 1, 6, 64)
    # sequence 1 runs over the end, sequence 2 starts before 0
    a.spec_kv4_append(k, k, _i32([0, 4, -2]), cache)
    rk, _ = a.spec_kv4_read(cache, _i32([0, 4, -2]), 4)
    torch.cuda.synchronize()
    got = rk.float().cpu().numpy()
    assert np.isnan(got[0, 1, 0, 16:32]).all()
    assert np.isfinite(got[0, 1, 0, :16]).all()
    assert got[0, 2, 0, 3] == -6 * 448
    assert (got[1, :2] != 0).all() and (got[1, 2:] == 0).all()
    assert (got[2, :2] == 0).all() and (got[2, 2:] != 0).all()
    assert (cache.k[1, :, :4] == 0).all() and (cache.k[2, :, 2:] == 0).all()


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("N,Hq,Hkv,prefix", [
    (1, 4, 4, [0, 5]),              # one row per head, no prefix at all
    (1, 32, 8, [700, 31]),          # single-token decoding
    (1, 8, 1, [255, 256, 257]),     # eight rows, tile borders
    (2, 5, 1, [33, 64]),            # ten rows
    (1, 16, 1, [1000, 3]),          # sixteen rows
    (7, 8, 2, [1, 63]),
    (16, 4, 1, [64, 65]),
    (60, 16, 4, [130, 0]),          # 240 rows, a tree-only sequence
    (64, 2, 2, [200, 191]),         # full mask words
    (33, 6, 3, [127, 129]),
    (27, 14, 2, [95, 300]),         # 189 rows, seven per head
    (64, 16, 2, [190, 40]),         # 512 rows: two CTAs a head
    (5, 8, 1, [64, 255]),           # forty rows
])
def test_tree_attention_kv4_matches_oracle(N, Hq, Hkv, prefix, D):
    B = len(prefix)
    S = max(prefix) + N + 9
    rng = np.random.default_rng(N * 100 + Hq + D)
    cache, vals = make_cache(N + D, B, Hkv, S, D,
                             used=[p + N for p in prefix])
    q = torch.randn(B, N, Hq, D, generator=_gen(N), device="cuda").bfloat16()
    _, words = tree_mask(random_parent(rng, B, N))
    out, lse = api().spec_tree_attention_kv4(
        q, cache, _i32(prefix), _words(words), scale=0.11, v_unit=0.125,
        lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, q, vals, prefix, words, 0.11)


@pytest.mark.parametrize("N,Hq,Hkv,B,lo,hi", [
    (1, 8, 2, 40, 0, 900),        # many ragged sequences, pieces cut units
    (1, 4, 2, 300, 0, 90),        # more sequences than threads
    (1, 4, 1, 1, 20000, 20000),   # one long sequence over many pieces
    (20, 8, 2, 3, 1500, 5000),    # tree rows over long ragged prefixes
    (60, 4, 1, 2, 2000, 6000),    # 240 rows, shares of a long prefix joined
    (6, 4, 1, 1, 30000, 30000),   # 24 rows over many pieces
])
def test_ragged_batches_and_split_sequences(N, Hq, Hkv, B, lo, hi):
    rng = np.random.default_rng(B + hi)
    prefix = rng.integers(lo, hi + 1, size=B)
    D, S = 128, int(prefix.max()) + N
    cache, vals = make_cache(B, B, Hkv, S, D)
    q = torch.randn(B, N, Hq, D, generator=_gen(B), device="cuda").bfloat16()
    _, words = tree_mask(random_parent(rng, B, N))
    out, lse = api().spec_tree_attention_kv4(
        q, cache, _i32(prefix), _words(words), v_unit=0.125, lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, q, vals, prefix, words, 128 ** -0.5)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("prefix", [[400, 33], [20001]])   # one CTA cluster; pieces
@pytest.mark.parametrize("N,Hq", [(1, 17), (1, 23), (3, 8), (5, 5), (31, 1),
                                  (4, 8), (3, 11), (2, 12)])
def test_rows_at_the_borders_of_row_tiles(N, Hq, prefix, D):
    rng = np.random.default_rng(N * Hq + D)
    B, S = len(prefix), max(prefix) + N + 1
    cache, vals = make_cache(N * Hq, B, 1, S, D)
    q = torch.randn(B, N, Hq, D, generator=_gen(Hq), device="cuda").bfloat16()
    _, words = tree_mask(random_parent(rng, B, N))
    out, lse = api().spec_tree_attention_kv4(
        q, cache, _i32(prefix), _words(words), v_unit=0.125, lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, q, vals, prefix, words, D ** -0.5)


def test_large_and_small_query_rows_and_units():
    # rows of very different magnitude, among them zeros; unit 2^-20 keys
    B, N, Hq, Hkv, D, P = 1, 3, 4, 2, 128, 150
    cache, vals = make_cache(2, B, Hkv, P + N, D, k_unit=2.0 ** -20,
                             v_unit=2.0 ** 10)
    q = torch.randn(B, N, Hq, D, generator=_gen(2), device="cuda")
    mag = torch.tensor([0.0, 1e-6, 1.0, 3e4, 1e-30, 7.0, 1e6, 0.01, 5.0, 2.0,
                        0.5, 100.0], device="cuda").reshape(B, N, Hq, 1)
    q = (q * mag).bfloat16()
    words = [[1, 3, 7]]
    out, lse = api().spec_tree_attention_kv4(
        q, cache, _i32([P]), _words(words), scale=0.5, k_unit=2.0 ** -20,
        v_unit=2.0 ** 10, lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, q, vals, [P], words, 0.5)


@pytest.mark.parametrize("N", [1, 2, 4, 10, 40])   # 8 to 320 rows
@pytest.mark.parametrize("D", [64, 128])
def test_growing_scores_rescale(N, D):
    # keys ordered so that the running maximum grows again and again
    B, Hq, Hkv, P = 1, 8, 1, 1500
    cache, vals = make_cache(4, B, Hkv, P + N, D)
    order = np.concatenate([np.argsort(vals[0][0, 0, :P].sum(-1)),
                            np.arange(P, P + N)])
    cache = api().KV4Cache(*[t[:, :, torch.from_numpy(order).cuda()].contiguous()
                             for t in cache])
    vals = tuple(x[:, :, order] for x in vals)
    q = torch.ones(B, N, Hq, D, device="cuda")
    q *= torch.linspace(0.25, 1.5, N * Hq, device="cuda").reshape(1, N, Hq, 1)
    q = q.bfloat16()
    words = [[(1 << (i + 1)) - 1 for i in range(N)]]
    out, lse = api().spec_tree_attention_kv4(
        q, cache, _i32([P]), _words(words), scale=2.0, v_unit=0.125, lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, q, vals, [P], words, 2.0)


def test_rows_that_see_nothing_and_clamped_prefix():
    B, N, Hq, Hkv, D, S = 3, 5, 4, 2, 128, 40
    cache, vals = make_cache(9, B, Hkv, S, D)
    q = torch.randn(B, N, Hq, D, generator=_gen(9), device="cuda").bfloat16()
    words = [[0, 1, 0, 8, 31], [1, 3, 5, 9, 17], [0] * 5]
    out, lse = api().spec_tree_attention_kv4(
        q, cache, _i32([0, 1000, -4]), _words(words), scale=0.1, v_unit=0.125,
        lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, q, vals, [0, S - N, 0], words, 0.1)
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    # mask bits at or above N do not count
    wide = [[w | (0x5 << N) for w in r] for r in words]
    again, _ = api().spec_tree_attention_kv4(
        q, cache, _i32([0, 1000, -4]), _words(wide), scale=0.1, v_unit=0.125)
    assert torch.equal(again, out)


@pytest.mark.parametrize("N,Hq,Hkv", [(6, 2, 2), (12, 4, 1), (20, 8, 2),
                                      (40, 8, 2)])
def test_nan_of_a_drafted_position_stays_on_its_branch(N, Hq, Hkv):
    D, P = 128, 70
    parent = np.array([[-1] + [max(0, (j - 1) // 2) for j in range(1, N)]])
    _, words = tree_mask(parent)
    cache, vals = make_cache(11, 1, Hkv, P + N, D)
    q = torch.randn(1, N, Hq, D, generator=_gen(3), device="cuda").bfloat16()
    args = (_i32([P]), _words(words))
    base, _ = api().spec_tree_attention_kv4(q, cache, *args)
    cache.v_scale[0, 0, P + 2, 3] = 0x7F       # dims 48 .. 63 of node 2
    cache.k_scale[0, Hkv - 1, P + 1, 0] = 0xFF  # node 1's key, another head
    out, _ = api().spec_tree_attention_kv4(q, cache, *args)
    torch.cuda.synchronize()
    G = Hq // Hkv
    want = base.float().cpu().numpy().copy()
    for i in range(N):
        if int(words[0][i]) >> 2 & 1:
            want[0, i, :G, 48:64] = np.nan
        if int(words[0][i]) >> 1 & 1:
            want[0, i, (Hkv - 1) * G:] = np.nan
    got = out.float().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(got[ok], want[ok])


def test_static_tree_workload_sampled_sequences():
    # the tree-attention workload's sizes; two sequences in full
    rng = np.random.default_rng(21)
    B, Hq, Hkv, D, S = 32, 32, 8, 128, 4096 + 64
    static = synth.static_tree(synth.workload("tree_static")).numpy()
    N = static.size
    _, words = tree_mask(np.tile(static, (B, 1)))
    prefix = rng.integers(2048, 4096, size=B).astype(np.int32)
    a = api()
    cache = a.kv4_cache(B, Hkv, S, D)
    g = _gen(23)
    k = torch.randn(B, S, Hkv, D, generator=g, device="cuda").bfloat16()
    v = torch.randn(B, S, Hkv, D, generator=g, device="cuda").bfloat16()
    a.spec_kv4_append(k, v, _i32([0] * B), cache)
    q = torch.randn(B, N, Hq, D, generator=g, device="cuda").bfloat16()
    out, lse = a.spec_tree_attention_kv4(q, cache, _i32(prefix),
                                         _words(words), lse=True)
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()
    for b in (0, 17):
        part = [t[b:b + 1].cpu().numpy() for t in cache]
        vals = (kv4.values(part[0], part[1]), kv4.values(part[2], part[3]))
        check_attention(out[b:b + 1], lse[b:b + 1], q[b:b + 1], vals,
                        prefix[b:b + 1], words[b:b + 1], 128 ** -0.5)


def test_repeats_are_bitwise_equal_and_graphs_replay():
    B, N, Hq, Hkv, D, S = 5, 3, 8, 2, 128, 2000
    cache, _ = make_cache(14, B, Hkv, S, D)
    q = torch.randn(B, N, Hq, D, generator=_gen(5), device="cuda").bfloat16()
    pre = _i32([1900, 3, 700, 1200, 64])
    words = _words([[1, 3, 5]] * B)
    a = api()
    first, l1 = a.spec_tree_attention_kv4(q, cache, pre, words, lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second, l2 = a.spec_tree_attention_kv4(q, cache, pre, words, lse=True,
                                           stream=s)
    s.synchronize()
    assert torch.equal(first, second) and torch.equal(l1, l2)
    with torch.cuda.stream(s):
        a.spec_tree_attention_kv4(q, cache, pre, words)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, l3 = a.spec_tree_attention_kv4(q, cache, pre, words, lse=True)
    pre.copy_(_i32([5, 1990, 0, 333, 1024]))
    q.copy_(q.flip(0))
    graph.replay()
    want, l4 = a.spec_tree_attention_kv4(q, cache, pre, words, lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(l3, l4)
