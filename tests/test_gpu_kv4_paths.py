"""Attention over the 4-bit cache and accumulated weights where the work of a
call is cut across sequences and heads: pieces of the line of key blocks that
end inside a unit, hold several whole ones, or pass from one head or sequence
to the next; joins found from the pieces' borders; more sequences than a scan
has threads; shares of a tree's blocks that hold none; weights' pieces of many
blocks.  Compared with the definition in float64 on the GPU, within the bounds
derived in test_gpu_kv4.py and test_gpu_evict.py.
"""

import math

import numpy as np
import pytest
import torch

from tests._parity import lib_ready
from tests.test_gpu_kv4 import _gen, _i32, api

pytestmark = pytest.mark.gpu

V_UNIT = 0.125
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def random_cache(g, B, Hkv, S, D):
    """Any codes, scales of 1/4 to 15/8."""
    u8 = lambda lo, hi, w: torch.randint(lo, hi, (B, Hkv, S, w), generator=g,
                                         device="cuda", dtype=torch.uint8)
    return api().KV4Cache(u8(0, 256, D // 2), u8(0x28, 0x40, D // 16),
                          u8(0, 256, D // 2), u8(0x28, 0x40, D // 16))


def values(codes, scales, unit):
    t = torch.tensor(CODES, dtype=torch.float64, device="cuda")
    t = torch.cat([t, -t])
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    s = scales.view(torch.float8_e4m3fn).double() * unit
    return t[c] * s.repeat_interleave(16, -1)


def random_words(rng, B, N):
    """Mask words of random trees, [B, N] int64 on the host."""
    w = np.zeros((B, N), dtype=np.uint64)
    for b in range(B):
        for j in range(N):
            up = -1 if j == 0 or rng.random() < 0.3 else int(rng.integers(0, j))
            w[b, j] = (w[b, up] if up >= 0 else np.uint64(0)) | np.uint64(1 << j)
    return torch.from_numpy(w.view(np.int64))


def check(out, lse, q, cache, prefix, words, scale):
    B, N, Hq, D = q.shape
    Hkv = cache.k.shape[1]
    G = Hq // Hkv
    for b in range(B):
        P = int(prefix[b])
        n = P + N
        k = values(cache.k[b, :, :n], cache.k_scale[b, :, :n], 1.0)
        v = values(cache.v[b, :, :n], cache.v_scale[b, :, :n], V_UNIT)
        qd = q[b].double().reshape(N, Hkv, G, D).permute(1, 0, 2, 3)
        qd = qd.reshape(Hkv, N * G, D)
        tree = (words[b].cuda().unsqueeze(1)
                >> torch.arange(N, device="cuda")) & 1
        see = torch.ones(N, n, dtype=torch.bool, device="cuda")
        see[:, P:] = tree.bool()
        see = see.repeat_interleave(G, 0)
        s = (qd @ k.transpose(1, 2) * scale).masked_fill(~see, -math.inf)
        norm = torch.logsumexp(s, -1)
        w = torch.exp(s - norm.unsqueeze(-1))
        ref = w @ v
        mag = (qd.abs() @ k.abs().transpose(1, 2) * scale
               ).masked_fill(~see, 0.0).amax(-1)
        e = mag * 2.0 ** -17
        A = w @ v.abs()
        ta = (2.0 ** -11 + 2 * e.unsqueeze(-1) + (n / 16 + 64) * 2.0 ** -23
              ) * A + n * 2.0 ** -32 * v.abs().max()
        rows = lambda x: x.reshape(N, Hkv, G, -1).transpose(0, 1).reshape(
            Hkv, N * G, -1)
        got = rows(out[b].double())
        err = (got - ref).abs() - ta - 2.0 ** -8 * ref.abs()
        assert torch.isfinite(got).all(), b
        assert float(err.max()) <= 0, (b, P, float(err.max()))
        rl = norm / math.log(2.0)
        tl = (math.log2(math.e) * (e + (n / 4 + 64) * 2.0 ** -24)
              + 2.0 ** -21 * (rl.abs() + 1))
        gl = rows(lse[b].double().unsqueeze(-1)).squeeze(-1)
        assert ((gl - rl).abs() <= tl).all(), (b, P)


def lengths(rng, B, most, short):
    """Short sequences, an empty one, and every eighth of any length."""
    p = rng.integers(0, short + 1, size=B)
    p[::8] = rng.integers(0, most + 1, size=p[::8].size)
    p[B // 3], p[-1] = 0, most
    return p


# Pieces of the line.  slack: what the caches hold beyond the longest sequence.
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("N,Hq,Hkv,B,most,short,slack", [
    # pieces end inside units, take several heads, pass to the next sequence
    (1, 8, 2, 24, 26000, 26000, 0),         # 4 rows a head
    (4, 8, 2, 20, 26000, 26000, 0),         # 16
    (5, 8, 2, 20, 12000, 12000, 7),         # 20
    (8, 4, 1, 20, 20000, 20000, 0),         # 32
    (1, 8, 1, 320, 2200, 300, 0),           # several sequences per scan thread
    (4, 4, 1, 460, 900, 200, 3500),         # the same, 16 rows, 384 threads
    # more units than borders between pieces: whole units beside cut ones
    (1, 8, 2, 1250, 2699, 150, 0),
    (4, 8, 2, 950, 2000, 150, 5000),
    (6, 8, 2, 640, 3000, 150, 1200),        # 24
    (16, 4, 2, 640, 3000, 150, 1200),       # 32
])
def test_pieces_of_ragged_batches(N, Hq, Hkv, B, most, short, slack, D):
    rng = np.random.default_rng(B + N)
    prefix = lengths(rng, B, most, short)
    S = most + N + slack
    # partial results: the call works on pieces, not on clusters per unit
    assert api()._kv4_workspace_bytes(B, N, Hq, Hkv, D, S) > 0
    g = _gen(B)
    cache = random_cache(g, B, Hkv, S, D)
    q = torch.randn(B, N, Hq, D, generator=g, device="cuda").bfloat16()
    words = random_words(rng, B, N)
    call = lambda: api().spec_tree_attention_kv4(
        q, cache, _i32(prefix), words.cuda(), v_unit=V_UNIT, lse=True)
    out, lse = call()
    again, l2 = call()
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, l2)
    check(out, lse, q, cache, prefix, words, D ** -0.5)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("N,Hq,Hkv,B,most,short,slack,split", [
    (40, 1, 1, 300, 333, 100, 0, False),    # more than are ordered by length
    (60, 4, 1, 260, 900, 300, 19000, True),  # most shares hold no block
    (20, 4, 2, 130, 900, 300, 19000, True),
    (60, 4, 1, 9, 70, 70, 4000, True),
])
def test_trees_in_many_sequences_and_empty_shares(N, Hq, Hkv, B, most, short,
                                                  slack, split, D):
    rng = np.random.default_rng(B + N)
    prefix = lengths(rng, B, most, short)
    S = most + N + slack
    assert (api()._kv4_workspace_bytes(B, N, Hq, Hkv, D, S) > 0) == split
    g = _gen(B)
    cache = random_cache(g, B, Hkv, S, D)
    q = torch.randn(B, N, Hq, D, generator=g, device="cuda").bfloat16()
    words = random_words(rng, B, N)
    call = lambda: api().spec_tree_attention_kv4(
        q, cache, _i32(prefix), words.cuda(), v_unit=V_UNIT, lse=True)
    out, lse = call()
    again, l2 = call()
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, l2)
    check(out, lse, q, cache, prefix, words, D ** -0.5)


# ------------------------------------------------------- accumulated weights
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("kind", ["kv4", "bf16"])
@pytest.mark.parametrize("N,Hq,Hkv,B,most,short", [
    (6, 32, 8, 16, 6000, 6000),     # five blocks and more a piece
    (40, 16, 4, 24, 5000, 5000),    # up to 160 rows: staged in parts per block
    (1, 8, 2, 700, 3000, 900),      # several sequences per scan thread
])
def test_weights_of_pieces_of_many_blocks(N, Hq, Hkv, B, most, short, kind, D):
    rng = np.random.default_rng(B + N)
    G, S, scale = Hq // Hkv, most + N + 3, D ** -0.5
    prefix = lengths(rng, B, most, short)
    lens = rng.integers(1, N + 1, size=B)
    nodes = np.stack([rng.permutation(N) for _ in range(B)]).astype(np.int32)
    lens[B // 3] = 0                 # an empty sequence without blocks
    lens[1], lens[5] = 0, N
    bad = [2, 3, 7]                  # invalid paths between valid ones
    lens[2], lens[3] = -1, N + 1
    nodes[7, 0], lens[7] = N, 1
    g = _gen(B)
    w0 = torch.rand(B, Hkv, S, generator=g, device="cuda")
    q = torch.randn(B, N, Hq, D, generator=g, device="cuda").bfloat16()
    if kind == "kv4":
        cache = random_cache(g, B, Hkv, S, D)
        kc = cache[:2]
        keys = lambda b, n: values(cache.k[b, :, :n], cache.k_scale[b, :, :n], 1.0)
    else:
        kc = torch.randn(B, Hkv, S, D, generator=g, device="cuda",
                         dtype=torch.bfloat16)
        keys = lambda b, n: kc[b, :, :n].double()
    lse = torch.zeros(B, N, Hq, device="cuda")
    ref = w0.double()
    tol = torch.zeros_like(ref)
    for b in range(B):
        if b in bad:
            continue
        P, n = int(prefix[b]), int(lens[b])
        ref[b, :, P:P + n] = 0
        k = keys(b, P + n)
        for t in range(n):
            L, i = P + t + 1, int(nodes[b, t])
            qd = q[b, i].double().reshape(Hkv, G, D)
            s = qd @ k[:, :L].transpose(1, 2) * (scale * math.log2(math.e))
            l = (torch.logsumexp(s * math.log(2.0), -1) / math.log(2.0)).float()
            lse[b, i] = l.reshape(Hq)
            l = l.double().unsqueeze(-1)
            mag = (qd.abs() @ k[:, :L].abs().transpose(1, 2)
                   * (scale * math.log2(math.e)))
            w = torch.exp2(s - l)
            e = (2.0 ** -17 * mag + 2.0 ** -23 * (mag + l.abs()) + 2.0 ** -22
                 + n * G * 2.0 ** -24)
            ref[b, :, :L] += w.sum(1)
            tol[b, :, :L] += (w * e).sum(1)
        tol[b, :, :P + n] += ref[b, :, :P + n].abs() * 2.0 ** -23
    out = w0.clone()
    api().spec_kv_weights(q, kc, lse, _i32(prefix), _i32(lens), _i32(nodes),
                          weights=out, out=out)
    torch.cuda.synchronize()
    err = (out.double() - ref).abs() - tol
    worst = int(err.flatten().argmax())
    assert float(err.max()) <= 0, (np.unravel_index(worst, err.shape),
                                   float(err.max()))
