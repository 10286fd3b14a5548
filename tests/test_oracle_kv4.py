"""Pins of the 4-bit cache, weight and eviction oracles (no GPU).

Pinned against torch's own float8_e4m3fn conversions, the bit fields of the
formats, brute force over all codes, and the tree-attention oracle."""

import numpy as np
import pytest
import torch

from oracle import evict, kv4
from oracle.attention import tree_attention
from oracle.tree import tree_mask


def test_tables_are_the_formats():
    b = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(kv4.E4M3, b.double().numpy())
    for c in range(8):  # sign, two exponent bits (bias 1), one mantissa bit
        e, m = c >> 1, c & 1
        assert kv4.E2M1[c] == (m * 0.5 if e == 0 else (1 + m / 2) * 2 ** (e - 1))


def test_scale_rounding_matches_torch_e4m3():
    x = torch.linspace(0, 447, 40001, dtype=torch.float32)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv4._nearest(x.double().numpy(), kv4.E4M3), want)


@pytest.mark.parametrize("unit", [1.0, 0.125, 4.0])
def test_codes_are_the_nearest(unit):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.normal(size=(40, 64)) * 3).bfloat16().double().numpy()
    codes, scales = kv4.quantise(x, unit)
    got = kv4.values(codes, scales, unit)
    s = np.repeat(kv4.E4M3[scales] * unit, 16, -1)
    grid = np.concatenate([-kv4.E2M1, kv4.E2M1])
    best = np.abs(x[..., None] - s[..., None] * grid).min(-1)
    assert np.allclose(np.abs(x - got), best, rtol=0, atol=1e-15)
    # a value already held in 4 bits comes back: the block maximum is 6 scales
    again = kv4.values(*kv4.quantise(got, unit), unit)
    full = np.abs(got).reshape(40, 4, 16).max(-1) == 6 * kv4.E4M3[scales] * unit
    assert np.array_equal(again.reshape(40, 4, 16)[full],
                          got.reshape(40, 4, 16)[full])


def test_ties_zero_blocks_and_special_values():
    x = np.zeros((1, 16))
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25]
    c, s = kv4.quantise(x)
    assert s[0, 0] == 0x38  # 1.0
    assert list(kv4.values(c, s)[0, :9]) == [6, 0, 1, 1, 2, 2, 4, 4, 0]
    c, s = kv4.quantise(np.zeros((1, 16)))
    assert s[0, 0] == 1 and (kv4.values(c, s) == 0).all()
    y = x.copy()
    y[0, 3] = np.nan
    assert np.isnan(kv4.values(*kv4.quantise(y))).all()
    y[0, 3] = np.inf
    assert kv4.values(*kv4.quantise(y))[0, 3] == 6 * 448


def test_attention_equals_the_tree_oracle():
    rng = np.random.default_rng(5)
    B, N, Hq, Hkv, D, S = 2, 6, 4, 2, 16, 15
    q = rng.normal(size=(B, N, Hq, D))
    k = rng.normal(size=(B, Hkv, S, D))
    v = rng.normal(size=(B, Hkv, S, D))
    parent = np.array([[-1, 0, 0, 1, -1, 4], [-1, 0, 1, 2, 3, 4]])
    _, bits = tree_mask(parent)
    out, lse = kv4.attention(q, k, v, [7, 0], bits, 0.3)
    assert np.allclose(out, tree_attention(q, k, v, [7, 0], parent, 0.3),
                       rtol=1e-13, atol=1e-13)
    # the normaliser turns scores into probabilities
    p = 2.0 ** (0.3 / np.log(2) * (k[0, 1, :8] @ q[0, 0, 2]) - lse[0, 0, 2])
    assert abs(p.sum() - 1) < 1e-12
    empty, l0 = kv4.attention(q, k, v, [0, 0], [[0] * N] * B, 0.3)
    assert (empty == 0).all() and np.isneginf(l0).all()


def test_weights_of_a_chain_are_softmax_columns():
    rng = np.random.default_rng(6)
    B, N, H, D, P = 1, 3, 2, 8, 5
    S = P + N
    q = rng.normal(size=(B, N, H, D))
    k = rng.normal(size=(B, H, S, D))
    words = [[(1 << (i + 1)) - 1 for i in range(N)]]
    _, lse = kv4.attention(q, k, k, [P], words, 0.5)
    out, lens = evict.add_weights(None, q, k, lse, [P], [2], None, 0.5)
    assert lens[0] == P + 2 and np.isnan(out[:, :, P + 2:]).all()
    for h in range(H):
        s0 = torch.softmax(torch.from_numpy(0.5 * k[0, h, :P + 1] @ q[0, 0, h]), 0)
        s1 = torch.softmax(torch.from_numpy(0.5 * k[0, h, :P + 2] @ q[0, 1, h]), 0)
        want = s1.numpy().copy()
        want[:P + 1] += s0.numpy()
        assert np.allclose(out[0, h, :P + 2], want, rtol=1e-12)
    # every row adds one per head
    assert np.allclose(np.nansum(out, -1), 2.0)
    bad, lens = evict.add_weights(None, q, k, lse, [P], [2],
                                  np.array([[0, 9, -1]]), 0.5)
    assert lens[0] == P and (bad[:, :, :P] == 0).all()


def test_kept_positions():
    w = np.array([0.0, 3, 1, 3, np.nan, 0, 9, 2])
    assert evict.kept_positions(w, 8, 4, 1) == [1, 3, 6, 7]
    assert evict.kept_positions(w, 8, 3, 2) == [1, 6, 7]    # tie: the lower
    assert evict.kept_positions(w, 8, 8, 2) == list(range(8))
    assert evict.kept_positions(w, 7, 6, 0) == [0, 1, 2, 3, 5, 6]
    assert evict.kept_positions(w, 8, 2, 2) == [6, 7]
    assert evict.kept_positions(np.zeros(6), 6, 3, 1) == [0, 1, 5]
    assert evict.kept_positions(w, -3, 4, 1) == []
