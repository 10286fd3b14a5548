"""Accumulated attention weights and eviction on the GPU vs the oracle.

Weights: a probability is 2^(x), x = f s - lse in float32.  With mag =
log2(e) scale sum_d |q_d k_d| the score errs by at most 2^-17 mag (see
test_gpu_kv4.py; bf16 caches multiply bf16 operands, also exact), the FMA by
2^-24 (|f s| + |lse|) <= 2^-23 (mag + |lse|), the exponential by 2^-22
relative; the sum over rows adds 2^-24 per term.  Eviction is exact.
"""

import numpy as np
import pytest
import torch

from oracle import evict, kv4
from oracle.kv import kv_commit
from oracle.tree import tree_mask
from tests._parity import lib_ready, np64
from tests.test_gpu_kv4 import (_gen, _i32, _words, api, check_attention,
                                make_cache, random_parent)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def _weight_bound(q, k, lse, prefix, lens, nodes, scale, ref, G):
    """Tolerance of the accumulated weights (rows as the oracle took them)."""
    tol = np.abs(ref) * 2.0 ** -23
    B, Hkv = ref.shape[:2]
    for b in range(B):
        P = int(prefix[b])
        n = lens[b] - P
        for t in range(n):
            i = t if nodes is None else int(nodes[b][t])
            for g in range(Hkv * G):
                if not np.isfinite(lse[b, i, g]):
                    continue
                h, L = g // G, P + t + 1
                s = scale * np.log2(np.e) * (k[b, h, :L] @ q[b, i, g])
                mag = scale * np.log2(np.e) * (np.abs(k[b, h, :L])
                                               @ np.abs(q[b, i, g]))
                w = 2.0 ** (s - lse[b, i, g])
                e = (2.0 ** -17 * mag + 2.0 ** -23 * (mag + abs(lse[b, i, g]))
                     + 2.0 ** -22)
                tol[b, h, :L] += w * (e + n * G * 2.0 ** -24)
    return tol


def _paths(rng, parent):
    B, N = parent.shape
    nodes = np.full((B, N), -1, dtype=np.int32)
    lens = np.zeros(B, dtype=np.int32)
    for b in range(B):
        cur = -1
        while True:
            kids = np.flatnonzero(parent[b] == cur)
            if kids.size == 0 or (lens[b] and rng.random() < 0.2):
                break
            cur = int(rng.choice(kids))
            nodes[b, lens[b]] = cur
            lens[b] += 1
    return nodes, lens


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("kind", ["kv4", "bf16"])
@pytest.mark.parametrize("N,Hq,Hkv,prefix", [
    (1, 4, 4, [0, 31, 1025]),
    (1, 16, 2, [1023, 5, 96]),
    (9, 8, 2, [100, 0, 2047]),
    (40, 12, 1, [64, 700, 3]),      # 12 heads on one: more rows than a stage
])
def test_weights_match_oracle(kind, N, Hq, Hkv, prefix, D):
    rng = np.random.default_rng(N * 10 + Hq + D)
    B, G = len(prefix), Hq // Hkv
    S = max(prefix) + N + 5
    parent = random_parent(rng, B, N)
    if N == 40:  # a chain: all 40 nodes accepted in one sequence
        parent[1] = np.arange(-1, N - 1)
    nodes, lens = _paths(rng, parent)
    if N == 40:
        nodes[1], lens[1] = np.arange(N), N
    q = torch.randn(B, N, Hq, D, generator=_gen(N), device="cuda").bfloat16()
    used = [p + int(n) for p, n in zip(prefix, lens)]
    if kind == "kv4":
        cache, (k, _) = make_cache(N, B, Hkv, S, D, used=used)
        kc = cache[:2]
    else:
        kc = torch.randn(B, Hkv, S, D, generator=_gen(D), device="cuda").bfloat16()
        k = np64(kc)
        for b in range(B):
            kc[b, :, used[b]:] = float("nan")
    # normalisers of the rows over what they see after the commit
    scale = 0.2
    lse = np.full((B, N, Hq), -np.inf)
    for b in range(B):
        for t in range(lens[b]):
            for h in range(Hq):
                s = scale * (k[b, h // G, :prefix[b] + t + 1]
                             @ np64(q)[b, nodes[b, t], h])
                lse[b, nodes[b, t], h] = np.log2(np.exp(s - s.max()).sum()
                                                 ) + s.max() * np.log2(np.e)
    lse32 = torch.from_numpy(lse).float()
    w0 = torch.rand(B, Hkv, S, generator=_gen(4), device="cuda")
    got = torch.full_like(w0, -7.0)
    args = (q, kc, lse32.cuda(), _i32(prefix), _i32(lens), _i32(nodes))
    api().spec_kv_weights(*args, scale=scale, weights=w0, out=got)
    torch.cuda.synchronize()
    ref, L = evict.add_weights(np64(w0), np64(q), k, lse32.double().numpy(),
                               prefix, lens, nodes, scale)
    tol = _weight_bound(np64(q), k, lse32.double().numpy(), prefix, L, nodes,
                        scale, np.nan_to_num(ref), G)
    g = got.double().cpu().numpy()
    for b in range(B):
        assert (g[b, :, L[b]:] == -7.0).all()   # behind the sequence
        assert (np.abs(g[b, :, :L[b]] - ref[b, :, :L[b]])
                <= tol[b, :, :L[b]]).all()
    # in place, and without a previous record
    w1 = w0.clone()
    api().spec_kv_weights(*args, scale=scale, weights=w1, out=w1)
    zero = api().spec_kv_weights(*args, scale=scale)
    torch.cuda.synchronize()
    for b in range(B):
        assert torch.equal(w1[b, :, :L[b]], got[b, :, :L[b]])
        assert torch.equal(w1[b, :, L[b]:], w0[b, :, L[b]:])
        assert (zero[b, :, L[b]:] == 0).all()
        new = slice(prefix[b], L[b])
        assert torch.equal(zero[b, :, new], got[b, :, new])


def test_weights_invalid_paths_and_empty_rows():
    B, N, Hq, Hkv, D, S = 5, 4, 2, 1, 64, 50
    cache, _ = make_cache(1, B, Hkv, S, D)
    q = torch.randn(B, N, Hq, D, generator=_gen(1), device="cuda").bfloat16()
    lse = torch.zeros(B, N, Hq, device="cuda")
    lse[4] = float("-inf")
    w0 = torch.rand(B, Hkv, S, device="cuda")
    nodes = _i32([[0, 1, -1, -1], [0, 4, -1, -1], [0, 1, 2, 3], [0] * 4,
                  [0, 1, 2, 3]])
    out = api().spec_kv_weights(q, cache[:2], lse, _i32([10, 10, 10, 10, 10]),
                                _i32([-1, 2, 5, 0, 2]), nodes, weights=w0,
                                out=w0.clone())
    torch.cuda.synchronize()
    assert torch.equal(out[:4], w0[:4])
    assert torch.equal(out[4, :, :10], w0[4, :, :10])
    assert (out[4, :, 10:12] == 0).all()
    assert torch.equal(out[4, :, 12:], w0[4, :, 12:])


# ------------------------------------------------------------------ evict
def _weights(rng, B, Hkv, S, kind):
    if kind == "ties":
        w = rng.integers(0, 4, size=(B, Hkv, S)).astype(np.float32)
    elif kind == "special":
        w = rng.normal(size=(B, Hkv, S)).astype(np.float32)
        pick = rng.random((B, Hkv, S))
        w[pick < 0.2] = np.nan
        w[(pick >= 0.2) & (pick < 0.3)] = -np.inf
        w[(pick >= 0.3) & (pick < 0.4)] = np.inf
        w[(pick >= 0.4) & (pick < 0.5)] = 0.0
        w[(pick >= 0.5) & (pick < 0.6)] = -0.0
        w[(pick >= 0.6) & (pick < 0.7)] = 1e-42
    else:
        w = np.exp(2 * rng.normal(size=(B, Hkv, S))).astype(np.float32)
    return w


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["plain", "ties", "special"])
@pytest.mark.parametrize("B,Hkv,S,length,budget,recent", [
    (1, 1, 1, [1], 1, 0),
    (2, 3, 40, [40, 17], 16, 16),
    (4, 2, 300, [300, 0, 16, 299], 16, 3),
    (3, 2, 1111, [1111, 700, 513], 512, 0),
    (1, 2, 9000, [8999], 7001, 640),
    (2, 1, 70001, [70001, 40000], 3001, 100),
    (1, 1, 131073, [131073], 4000, 7),       # a cluster of sixteen
    (1, 2, 262145, [262145], 60000, 60),     # more than a cluster holds
])
def test_evict_matches_oracle(B, Hkv, S, length, budget, recent, kind, in_place):
    rng = np.random.default_rng(S + budget)
    w = _weights(rng, B, Hkv, S, kind)
    if kind == "special":  # an index row decides among every NaN and -inf
        w[0, 0, :] = np.where(rng.random(S) < 0.5, np.nan, -np.inf)
    planes = [torch.randint(0, 256, (B, Hkv, S, r), dtype=torch.uint8,
                            device="cuda") for r in (64, 8, 5)]
    planes.append(torch.randn(B, Hkv, S, 3, 8, device="cuda").bfloat16())
    before = [p.cpu() for p in planes]
    wt = torch.from_numpy(w).cuda()
    a = api()
    if in_place:
        outs, wo, S_out = planes, wt, S
        kept, new_len = a.spec_kv_evict(wt, _i32(length), planes,
                                        budget=budget, recent=recent)
    else:
        S_out = budget + 3
        outs = [torch.zeros(B, Hkv, S_out, *p.shape[3:], dtype=p.dtype,
                            device="cuda") for p in planes]
        wo = torch.zeros(B, Hkv, S_out, device="cuda")
        kept, new_len = a.spec_kv_evict(wt, _i32(length), planes,
                                        budget=budget, recent=recent,
                                        planes_out=outs, weights_out=wo)
    torch.cuda.synchronize()
    assert new_len.tolist() == [min(n, budget) for n in length]
    kept = kept.cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            want = evict.kept_positions(w[b, h], length[b], budget, recent)
            n = len(want)
            assert kept[b, h, :n].tolist() == want
            assert (kept[b, h, n:] == -1).all()
            for p, o in zip(before, outs):
                assert torch.equal(o[b, h, :n].cpu(), p[b, h, want])
                tail = p[b, h, n:] if in_place else torch.zeros_like(
                    o[b, h, n:]).cpu()
                assert torch.equal(o[b, h, n:].cpu(), tail)
            assert np.array_equal(wo[b, h, :n].cpu().numpy(), w[b, h, want],
                                  equal_nan=True)


@pytest.mark.parametrize("B", [7, 20, 40])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_batches_match_oracle(B, in_place):
    # few and many (sequence, head) pairs: chunks of 1024, 512, 256 threads
    length = [(37 * b) % 1291 for b in range(B)]
    test_evict_matches_oracle(B, 2, 1290, length, 700, 31, "plain", in_place)


@pytest.mark.parametrize("S", [512, 513, 1024, 1537, 16384, 16385, 90000])
@pytest.mark.parametrize("bits", [7, 8, 15, 16, 23, 24, 31])
def test_evict_where_the_key_is_decided_early(S, bits):
    """The heavier group's keys differ from the others' first in the given bit
    from the top, so a select by digits can stop, or must go on, after any of
    them; runs of whole and broken lengths."""
    rng = np.random.default_rng(S + bits)
    heavy = rng.random(S) < 0.3
    low = (1 << (31 - bits)) - 1
    u = np.full(S, 0x3F200000 & ~((low << 1) | 1), np.uint32)
    u |= rng.integers(0, low + 1, size=S).astype(np.uint32)
    u[heavy] |= np.uint32(low + 1)
    w = u.view(np.float32)[None, None]
    a = api()
    n = int(heavy.sum())
    for budget in (n, n + 1, max(1, n - 1), max(1, n // 2)):
        t = torch.from_numpy(w.copy()).cuda()
        kept, _ = a.spec_kv_evict(t, _i32([S]), (), budget=budget, recent=0)
        torch.cuda.synchronize()
        want = evict.kept_positions(w[0, 0], S, budget, 0)
        assert kept[0, 0].tolist() == want
        assert np.array_equal(t[0, 0, :budget].cpu().numpy(), w[0, 0, want])


def test_evict_without_planes_and_empty_batch():
    a = api()
    w = torch.tensor([[[3.0, 1.0, 2.0, 0.0]]], device="cuda")
    kept, n = a.spec_kv_evict(w, _i32([4]), (), budget=2, recent=1)
    assert kept.tolist() == [[[0, 3]]] and n.tolist() == [2]
    assert w[0, 0, :2].tolist() == [3.0, 0.0]
    z = torch.empty(0, 2, 8, device="cuda")
    kept, n = a.spec_kv_evict(z, torch.empty(0, dtype=torch.int32,
                                             device="cuda"), (),
                              budget=2, recent=1)
    assert kept.shape == (0, 2, 2) and n.numel() == 0


# -------------------------------------------------- the operators together
def test_a_verification_step_on_an_evicted_4_bit_cache():
    """append -> attention -> commit -> weights -> evict -> attention, each
    checked against the oracle run on what the step before returned."""
    rng = np.random.default_rng(8)
    B, N, Hq, Hkv, D, S = 3, 12, 8, 2, 128, 400
    G, scale = Hq // Hkv, 128 ** -0.5
    a = api()
    g = _gen(8)
    pre = [300, 12, 257]
    cache = a.kv4_cache(B, Hkv, S, D)
    mk = lambda n: [torch.randn(B, n, Hkv, D, generator=g, device="cuda"
                                ).bfloat16() for _ in range(2)]
    a.spec_kv4_append(*mk(300), _i32([0] * B), cache)
    weights = torch.rand(B, Hkv, S, generator=g, device="cuda")
    for step in range(2):
        parent = random_parent(rng, B, N)
        _, words = tree_mask(parent)
        nodes, lens = _paths(rng, parent)
        q = torch.randn(B, N, Hq, D, generator=g, device="cuda").bfloat16()
        tpre = _i32(pre)
        a.spec_kv4_append(*mk(N), tpre, cache)
        out, lse = a.spec_tree_attention_kv4(q, cache, tpre, _words(words),
                                             lse=True)
        torch.cuda.synchronize()
        host = [t.cpu().numpy() for t in cache]
        vals = (kv4.values(host[0], host[1]), kv4.values(host[2], host[3]))
        check_attention(out, lse, q, vals, pre, words, scale)
        for t in cache:  # the accepted path's rows, plane by plane
            row = t.shape[-1]
            new_len = a.spec_kv_commit(
                t, tpre, _i32(lens), _i32(nodes), row_bytes=row, N=N,
                layout=(1, Hkv, Hkv * S * row, 0, S * row, row))
        torch.cuda.synchronize()
        host = [kv_commit(x.transpose(0, 2, 1, 3), pre, lens, nodes)[0]
                .transpose(0, 2, 1, 3) for x in host]
        for t, x in zip(cache, host):
            assert np.array_equal(t.cpu().numpy(), x)
        k = kv4.values(host[0], host[1])
        w0 = np64(weights)
        a.spec_kv_weights(q, cache, lse, tpre, _i32(lens), _i32(nodes),
                          weights=weights, out=weights)
        torch.cuda.synchronize()
        l64 = lse.double().cpu().numpy()
        ref, L = evict.add_weights(w0, np64(q), k, l64, pre, lens, nodes, scale)
        tol = _weight_bound(np64(q), k, l64, pre, L, nodes, scale,
                            np.nan_to_num(ref), G)
        got = np64(weights)
        assert L.tolist() == new_len.tolist()
        for b in range(B):
            assert (np.abs(got[b, :, :L[b]] - ref[b, :, :L[b]])
                    <= tol[b, :, :L[b]]).all()
        w32 = weights.cpu().numpy()
        kept, nl = a.spec_kv_evict(weights, new_len, cache, budget=100,
                                   recent=30)
        torch.cuda.synchronize()
        pre = nl.tolist()
        for b in range(B):
            for h in range(Hkv):
                want = evict.kept_positions(w32[b, h], int(L[b]), 100, 30)
                assert kept[b, h, :len(want)].tolist() == want
                for t, x in zip(cache, host):
                    assert np.array_equal(t[b, h, :len(want)].cpu().numpy(),
                                          x[b, h, want])


def test_eviction_replays_in_a_graph():
    B, Hkv, S, D = 2, 2, 600, 64
    cache, _ = make_cache(5, B, Hkv, S, D)
    a = api()
    w = torch.rand(B, Hkv, S, generator=_gen(6), device="cuda")
    n = _i32([600, 580])
    out = a.kv4_cache(B, Hkv, 128, D)
    wo = torch.zeros(B, Hkv, 128, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda: a.spec_kv_evict(w, n, cache, budget=128, recent=16,
                                   planes_out=out, weights_out=wo)
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept, new_len = call()
    w.copy_(w.flip(-1))
    n.copy_(_i32([99, 600]))
    graph.replay()
    torch.cuda.synchronize()
    moved = [t.clone() for t in out]
    wh = w.cpu().numpy()
    for b, h in ((0, 0), (0, 1), (1, 0), (1, 1)):
        want = evict.kept_positions(wh[b, h], int(n[b]), 128, 16)
        assert kept[b, h, :len(want)].tolist() == want
        for t, o in zip(cache, moved):
            assert torch.equal(o[b, h, :len(want)], t[b, h, want])


@pytest.mark.parametrize("N,Hq,Hkv,prefix", [
    (1, 4, 4, [0, 5]), (7, 8, 2, [1, 63]), (60, 16, 4, [130, 0]),
    (33, 6, 3, [127, 129])])
def test_bf16_attention_returns_its_normalisers(N, Hq, Hkv, prefix):
    """spec_tree_attention_lse: out bit for bit spec_tree_attention's; lse the
    oracle's within 2^-14 of the score magnitudes (float32 sums of 128
    products at 2^-24 each, doubled) and 2^-18 for the sum and the logarithm;
    then the weights of a bf16 cache sum to one per accepted row and head
    (within the same bounds, 2^-12 relative here)."""
    B, D = len(prefix), 128
    S = max(prefix) + N + 9
    rng = np.random.default_rng(N)
    g = _gen(N)
    q = torch.randn(B, N, Hq, D, generator=g, device="cuda").bfloat16()
    k = torch.randn(B, Hkv, S, D, generator=g, device="cuda").bfloat16()
    v = torch.randn(B, Hkv, S, D, generator=g, device="cuda").bfloat16()
    parent = random_parent(rng, B, N)
    parent[0] = np.arange(-1, N - 1)     # a chain in sequence 0
    _, words = tree_mask(parent)
    pre = _i32(prefix)
    a = api()
    base = a.spec_tree_attention(q, k, v, pre, _words(words), scale=0.09)
    out, lse = a.spec_tree_attention_lse(q, k, v, pre, _words(words),
                                         scale=0.09)
    torch.cuda.synchronize()
    assert torch.equal(out, base)
    _, ref = kv4.attention(np64(q), np64(k), np64(v), prefix, words, 0.09)
    mag = 0.09 * np.abs(np64(q)).sum(-1) * np.abs(np64(k)).max()
    err = np.abs(lse.double().cpu().numpy() - ref)
    assert (err <= 2.0 ** -14 * mag + 2.0 ** -18 * (1 + np.abs(ref))).all()
    # sequence 0's chain is accepted whole, the others' nothing
    lens = _i32([N] + [0] * (B - 1))
    w = a.spec_kv_weights(q, k, lse, pre, lens, scale=0.09)
    torch.cuda.synchronize()
    total = w[0].double().sum(-1).cpu().numpy()
    want = N * (Hq // Hkv)
    assert np.allclose(total, want, rtol=2.0 ** -12)
    assert (w[1:] == 0).all()


def test_calls_on_two_streams_at_once():
    """Every operator with a stream of its own, two sets in flight at the same
    time, equal to the same calls one after the other."""
    a = api()
    N, Hq, Hkv, D, S = 3, 8, 2, 128, 5000

    def step(seed, stream):
        g = _gen(seed)
        mk = lambda n, h: torch.randn(1, n, h, D, generator=g, device="cuda"
                                      ).bfloat16()
        k, v, q = mk(S - 10, Hkv), mk(S - 10, Hkv), mk(N, Hq)
        pre = _i32([S - 10 - N])
        words = _words([[1, 3, 5]])
        cache = a.kv4_cache(1, Hkv, S, D)
        small = a.kv4_cache(1, Hkv, 512, D)
        zero, lens = _i32([0]), _i32([2])
        torch.cuda.synchronize()
        for _ in range(3):
            a.spec_kv4_append(k, v, zero, cache, stream=stream)
            out, lse = a.spec_tree_attention_kv4(q, cache, pre, words, lse=True,
                                                 stream=stream)
            w = a.spec_kv_weights(q, cache, lse, pre, lens, stream=stream)
            kept, n = a.spec_kv_evict(w, pre, cache, budget=512, recent=100,
                                      planes_out=small, stream=stream)
            rk, rv = a.spec_kv4_read(small, zero, 512, stream=stream)
        return out, lse, w, kept, n, rk, rv

    s = [torch.cuda.Stream() for _ in range(2)]
    both = [step(i, s[i]) for i in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        alone = step(i, s[i])
        torch.cuda.synchronize()
        for x, y in zip(both[i], alone):
            assert torch.equal(x, y)


def test_views_and_host_tensors_are_refused():
    a = api()
    cache = a.kv4_cache(1, 2, 64, 128)
    k = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    z = _i32([0])
    with pytest.raises(ValueError, match="contiguous"):
        a.spec_kv4_append(k.transpose(1, 2).contiguous().transpose(1, 2), k, z,
                          cache)
    with pytest.raises(ValueError):
        a.spec_kv4_append(k, k, z.cpu(), cache)
    w = torch.zeros(1, 2, 64, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        a.spec_kv_evict(w.transpose(1, 2).contiguous().transpose(1, 2), z,
                        cache, budget=4, recent=0)
    from speculative_decoding_verification_tree_gb300 import SpecError
    with pytest.raises(SpecError):
        a.spec_kv_evict(w, z, cache, budget=65, recent=0)   # more than S
    with pytest.raises(SpecError):
        a.spec_kv_evict(w, z, cache, budget=4, recent=0, new_len=z)
    with pytest.raises(SpecError):
        a.spec_kv4_append(k, k, z, cache, k_unit=0.3)


def test_evict_takes_a_buffer_in_place_and_as_another_input():
    """A plane moved in place and copied by the same call, and the weights
    moved as a plane of their own, below and above what a cluster holds."""
    a = api()
    for S in (900, 262145):
        g = _gen(S)
        w = torch.rand(1, 2, S, generator=g, device="cuda")
        k = torch.randint(0, 256, (1, 2, S, 8), generator=g, device="cuda",
                          dtype=torch.uint8)
        w0, k0 = w.clone(), k.clone()
        copy = torch.zeros(1, 2, S, 8, dtype=torch.uint8, device="cuda")
        kept, n = a.spec_kv_evict(w, _i32([S]), (k, k, w), budget=300,
                                  recent=20, planes_out=(k, copy, w))
        torch.cuda.synchronize()
        assert n.tolist() == [300]
        for h in range(2):
            want = evict.kept_positions(w0[0, h].cpu().numpy(), S, 300, 20)
            assert kept[0, h].tolist() == want
            for got, src in ((w, w0), (k, k0), (copy, k0)):
                assert torch.equal(got[0, h, :300], src[0, h, want])
