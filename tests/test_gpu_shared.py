"""Tree attention over shared prefixes on the GPU vs the oracle.

Tolerances as in test_gpu_prompt.py, with n all keys a row can see; the join of
up to 152 pieces of two tiles adds as many float32 steps: (n / 16 + 400) 2^-23 A
for outputs and 400 more 2^-24 for normalisers.
"""

import numpy as np
import pytest
import torch

from oracle import shared as oracle
from tests._parity import lib_ready, np64
from tests.test_gpu_kv4 import random_parent

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def api():
    from speculative_decoding_verification_tree_gb300 import api as a
    return a


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def words(bits):
    return torch.from_numpy(np.asarray(bits, dtype=np.uint64).view(np.int64)
                            ).cuda()


def tree_bits(seed, B, N):
    from oracle.tree import tree_mask
    return tree_mask(random_parent(np.random.default_rng(seed), B, N))[1]


class Case:
    """Inputs; what lies behind the used positions is NaN."""

    def __init__(self, slen, start, pre, N, Hq, Hkv, D, seed=0, slack=3,
                 bits=None, std=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.B = B = len(pre)
        Sp, S = max(slen) + slack, max(pre) + N + slack
        rnd = lambda *s: (torch.randn(*s, D, generator=g, device="cuda")
                          * std).bfloat16()
        self.q = rnd(B, N, Hq)
        self.kp, self.vp = rnd(len(slen), Hkv, Sp), rnd(len(slen), Hkv, Sp)
        self.k, self.v = rnd(B, Hkv, S), rnd(B, Hkv, S)
        for t, lens, more in ((self.kp, slen, 0), (self.vp, slen, 0),
                              (self.k, pre, N), (self.v, pre, N)):
            for i, n in enumerate(lens):
                t[i, :, n + more:] = float("nan")
        self.slen, self.start, self.pre = slen, start, pre
        self.bits = tree_bits(seed, B, N) if bits is None else bits
        self.scale = D ** -0.5

    def args(self):
        return (self.q, self.kp, self.vp, i32(self.slen), i32(self.start),
                self.k, self.v, i32(self.pre), words(self.bits))

    def run(self, **kw):
        return api().spec_tree_attention_shared(*self.args(), scale=self.scale,
                                                lse=True, **kw)

    def want(self, only=None):
        return oracle.tree_attention_shared(
            np64(self.q), np64(self.kp), np64(self.vp), self.slen, self.start,
            np64(self.k), np64(self.v), self.pre, self.bits, self.scale)

    def check(self, out, lse):
        o, l, mag, sm = self.want()
        n = max(self.slen) + max(self.pre) + self.q.shape[1]
        e = 2.0 ** -17 * sm
        tol = (2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * e[..., None]
               + (n / 16 + 400) * 2.0 ** -23) * mag + 1e-30)
        live = ~np.isnan(l)
        err = np.abs(np64(out) - o)
        assert (err <= tol)[live].all(), float((err / tol)[live].max())
        g, inf = np64(lse), np.isneginf(l)
        assert np.isneginf(g[inf]).all()
        tl = 1.4427 * (e + (n / 4 + 400) * 2.0 ** -24) + 2.0 ** -21 * np.abs(l)
        ok = live & ~inf
        assert (np.abs(g - np.where(ok, l, 0)) <= tl)[ok].all()


CASES = [  # shared lengths, group starts, own prefixes, N, Hq, Hkv
    ([1], [0, 1], [0], 1, 1, 1),
    ([0], [0, 2], [0, 5], 1, 8, 2),
    ([128], [0, 3], [0, 127, 128], 1, 8, 2),
    ([1000], [0, 5], [0, 1, 64, 300, 129], 1, 8, 2),
    ([5000], [0, 2], [10, 900], 1, 32, 8),          # cut into many pieces
    ([300], [0, 40], list(range(40)), 1, 8, 2),     # 160 rows: two tiles
    ([300], [0, 70], list(range(70)), 1, 8, 1),     # several units a prefix
    ([700, 0, 129], [0, 3, 3, 7], [5, 70, 200, 0, 1, 2, 3], 7, 14, 2),
    ([260, 511], [0, 1, 4], [33, 128, 0, 400], 60, 8, 2),   # 240 rows
    ([260], [0, 2], [33, 140], 64, 32, 2),          # units share a sequence
    ([130], [0, 2], [3, 140], 3, 128, 1),
    ([400], [0, 3], [100, 2, 50], 20, 5, 5),
    ([64, 65, 66, 67], [0, 1, 2, 3, 4], [1, 2, 3, 4], 5, 65, 1),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[3:]}")
@pytest.mark.parametrize("D", [128, 64])
def test_shapes(case, D):
    c = Case(*case, D, seed=case[3])
    c.check(*c.run())


def test_long_prefix_many_samples():
    c = Case([9000], [0, 24], list(range(0, 240, 10)), 1, 8, 2, 128, seed=2)
    c.check(*c.run())
    c = Case([4100], [0, 3], [300, 0, 129], 33, 4, 1, 64, seed=3)
    c.check(*c.run())


def test_equals_the_call_without_sharing():
    """The same keys as one cache: what spec_tree_attention_lse gives, within
    both calls' tolerance (twice that of the oracle's)."""
    B, N, P = 4, 12, 200
    c = Case([500], [0, B], [P] * B, N, 8, 2, 128, seed=4)
    out, lse = c.run()
    cat = lambda x, y: torch.cat([x[:, :, :500].expand(B, -1, -1, -1),
                                  y[:, :, :P + N]], 2).contiguous()
    o2, l2 = api().spec_tree_attention_lse(
        c.q, cat(c.kp, c.k), cat(c.vp, c.v), i32([500 + P] * B), words(c.bits))
    o, l, mag, sm = c.want()
    tol = 2 * (2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -16 * sm[..., None]
               + 500 * 2.0 ** -23) * mag)
    assert (np.abs(np64(out) - np64(o2)) <= tol).all()
    assert (np.abs(np64(lse) - np64(l2)) <= 2.0 ** -15 * (sm + 1)).all()


def test_rows_that_see_nothing_and_sequences_outside():
    B, N = 6, 4
    bits = np.zeros((B, N), dtype=np.uint64)
    bits[3, 2] = 1 << 2
    c = Case([0, 40], [1, 4, 5], [0, 0, 3, 0, 2, 1], N, 4, 2, 128, seed=5,
             bits=bits)
    out = torch.full(c.q.shape, 7.0, device="cuda").bfloat16()
    lse = torch.full(c.q.shape[:3], 7.0, device="cuda")
    api().spec_tree_attention_shared(*c.args(), scale=c.scale, out=out, lse=lse)
    c.check(out, lse)
    for b in (0, 5):
        assert (out[b] == 7).all() and (lse[b] == 7).all()
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert (out[3, [0, 1, 3]] == 0).all() and torch.isneginf(lse[3, 0]).all()
    assert torch.equal(out[3, 2, :2], c.v[3, 0, 2].expand(2, -1))


def test_lengths_are_clamped():
    c = Case([90], [0, 3], [40, 7, 20], 5, 8, 2, 64, seed=6)
    want = c.run()
    a = list(c.args())
    c2 = Case([90], [0, 3], [40, 7, 20], 5, 8, 2, 64, seed=6, slack=0)
    a2 = list(c2.args())
    base = c2.run()
    a2[3], a2[4], a2[7] = i32([999]), i32([-4, 77]), i32([1000, 7, 20])
    got = api().spec_tree_attention_shared(*a2, scale=c.scale, lse=True)
    assert all(torch.equal(x, y) for x, y in zip(got, base))
    a[7] = i32([-3, 7, 20])
    got = api().spec_tree_attention_shared(*a, scale=c.scale, lse=True)
    assert torch.equal(got[0][1:], want[0][1:])
    c.pre[0] = 0
    assert torch.isfinite(got[0]).all()


@pytest.mark.parametrize("slen", [700, 7000])
@pytest.mark.parametrize("D", [128, 64])
def test_nan_and_infinity_reach_only_rows_that_see_them(slen, D):
    """In one sequence's own keys, in a drafted node, in the shared prefix; in
    pieces (long prefix) and units that are not cut."""
    B, N = 5, 6
    c = Case([slen], [0, B], [50, 0, 130, 300, 7], N, 8, 2, D, seed=7)
    base, lse0 = c.run()
    norm = lambda t: torch.nan_to_num(t, 77., 88., 99.)
    for b, pos in ((0, 3), (2, 128), (3, 299)):
        for val in (float("nan"), float("inf"), -float("inf")):
            keep = c.v[b, 1, pos, 5].clone()
            c.v[b, 1, pos, 5] = val
            out, lse = c.run()
            c.v[b, 1, pos, 5] = keep
            want = base.clone()
            want[b, :, 4:, 5] = val
            assert torch.equal(norm(out), norm(want)) and torch.equal(lse, lse0)
        keep = c.k[b, 0, pos, 9].clone()
        c.k[b, 0, pos, 9] = float("nan")
        out, lse = c.run()
        c.k[b, 0, pos, 9] = keep
        want = base.clone()
        want[b, :, :4] = float("nan")
        assert torch.equal(norm(out), norm(want))
        assert torch.isnan(lse[b, :, :4]).all()
    for b, j in ((1, 2), (4, 5)):       # a node's value: rows that see it
        pos = c.pre[b] + j
        keep = c.v[b, 0, pos, 0].clone()
        c.v[b, 0, pos, 0] = float("inf")
        out, _ = c.run()
        c.v[b, 0, pos, 0] = keep
        want = base.clone()
        for i in range(N):
            if (int(c.bits[b, i]) >> j) & 1:
                want[b, i, :4, 0] = float("inf")
        assert torch.equal(norm(out), norm(want))
    for pos in (0, slen - 1):           # the prefix: every sequence
        keep = c.vp[0, 1, pos, 2].clone()
        c.vp[0, 1, pos, 2] = float("nan")
        out, _ = c.run()
        c.vp[0, 1, pos, 2] = keep
        want = base.clone()
        want[:, :, 4:, 2] = float("nan")
        assert torch.equal(norm(out), norm(want))


def test_moving_maxima_across_pieces():
    """Scores that grow towards either end of a long prefix."""
    for sign in (1, -1):
        c = Case([6000], [0, 3], [100, 5, 0], 2, 8, 2, 128, seed=8)
        ramp = torch.linspace(-1, 1, 6003, device="cuda")[:, None] * sign
        c.kp = (c.kp.float() * 0.1 + ramp * 4).bfloat16()
        c.q = (c.q.float() * 0.1 + 2).bfloat16()
        c.scale = 1.0
        c.check(*c.run())


def test_many_sequences_and_prefixes():
    rng = np.random.default_rng(9)
    B, n = 900, 256
    start = np.sort(rng.integers(0, B + 1, size=n + 1))
    start[0], start[-1] = 0, B
    c = Case(rng.integers(0, 200, size=n).tolist(), start.tolist(),
             rng.integers(0, 30, size=B).tolist(), 1, 2, 1, 64, seed=10)
    c.check(*c.run())


def test_far_positions_pass_32_bits():
    """Prefixes and caches past 2^31 elements."""
    Hkv, Sp, D = 8, 1 << 21, 128     # 2 x 8 x 2^21 x 128 = 2^32 elements
    kp = torch.zeros(2, Hkv, Sp, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    n = 300
    for t in (kp, vp):
        t[1, 7, :n] = torch.randn(n, D, generator=g, device="cuda")
    c = Case([4, n], [0, 0, 2], [5, 200], 3, 8, 8, D, seed=12, slack=0)
    c.kp[1, 7, :n], c.vp[1, 7, :n] = kp[1, 7, :n], vp[1, 7, :n]
    small = c.run()
    c.kp, c.vp = kp, vp
    big = c.run()
    assert torch.equal(big[0][:, :, 7], small[0][:, :, 7])
    assert torch.equal(big[1][:, :, 7], small[1][:, :, 7])


def test_streams_graphs_and_equal_bits():
    c = Case([3000], [0, 6], [10, 50, 0, 7, 300, 90], 4, 16, 4, 128, seed=13)
    base = c.run()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(base, c.run()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.run(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(base, other))
    a = c.args()
    call = lambda: api().spec_tree_attention_shared(*a, scale=c.scale, lse=True)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = call()
    with torch.cuda.graph(g2):
        o2 = call()
    a[0].mul_(0.5)
    a[3].copy_(i32([2100]))
    g1.replay()
    g2.replay()
    want = call()
    for o in (o1, o2):
        assert all(torch.equal(x, y) for x, y in zip(o, want))
