"""Cases and plain forms of the 4-bit KV-cache and cache-eviction operators.

Four operators a decode loop with tree verification runs around its cache:

  append     the new positions' keys and values rounded into a 4-bit cache
             (e2m1 codes, one e4m3 scale per 16 head dims), and read back
  attention  tree / single-token attention over that cache, with the rows'
             log normalisers
  weights    attention weight received by every cached position, summed over
             the accepted rows and the query heads of a key/value head
  evict      the positions of highest accumulated weight and the most recent
             ones gathered into a smaller cache

`own` selects what `run` calls: the plain forms below (elementary torch
operations in float32) or the library's entry points.
"""

import math

import torch

own = False

LOG2E = 1.4426950408889634
BLOCK = 16                      # head dims that share one e4m3 scale
CODE_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one verification step's 60 drafted nodes of 32 sequences written
        # behind their prefixes (the library's static-tree workload)
        dict(name="append_tree_b32", op="append", B=32, n=60, Hkv=8, D=128,
             S=4160, lo=2048, hi=4095),
        # prompts of 8192 tokens written at once (prefill of four requests)
        dict(name="append_prefill_8k", op="append", B=4, n=8192, Hkv=8, D=128,
             S=8256, lo=0, hi=0),
        # a single user's short chat, one token: latency is everything
        dict(name="decode_b1_1k", op="attention", B=1, N=1, Hq=32, Hkv=8,
             D=128, S=1100, lo=1023, hi=1023),
        # plain decoding of a batch, ragged prefixes
        dict(name="decode_b32", op="attention", B=32, N=1, Hq=32, Hkv=8,
             D=128, S=4160, lo=2048, hi=4095),
        # one long document, one token at a time: few rows, a long axis
        dict(name="decode_b1_128k", op="attention", B=1, N=1, Hq=32, Hkv=8,
             D=128, S=131137, lo=131071, hi=131071),
        # a full server of long contexts: 2.4 GB of cache per call
        dict(name="decode_b64_32k", op="attention", B=64, N=1, Hq=32, Hkv=8,
             D=128, S=32832, lo=32000, hi=32767),
        # verification of 60-node trees (the library's tree-attention workload)
        dict(name="tree_b32", op="attention", B=32, N=60, Hq=32, Hkv=8, D=128,
             S=4160, lo=2048, hi=4095),
        # a small model's odd sizes: 27 nodes, 7 query heads per key/value
        # head, head dim 64, prefixes that end inside a tile
        dict(name="tree_odd_d64", op="attention", B=5, N=27, Hq=14, Hkv=2,
             D=64, S=5003, lo=17, hi=4931),
        # accumulated weights after a verification step on the 4-bit cache
        dict(name="weights_tree_b32", op="weights", cache="kv4", B=32, N=60,
             Hq=32, Hkv=8, D=128, S=4160, lo=2048, hi=4095),
        # the same bookkeeping in plain decoding over a bfloat16 cache
        dict(name="weights_decode_bf16", op="weights", cache="bf16", B=32,
             N=1, Hq=32, Hkv=8, D=128, S=4160, lo=2048, hi=4095),
        # a batch's caches cut to half: 4-bit planes
        dict(name="evict_b32_half", op="evict", cache="kv4", B=32, Hkv=8,
             D=128, S=4160, lo=2048, hi=4095, budget=2048, recent=256),
        # one long bfloat16 prompt cache compressed before decoding starts
        dict(name="evict_b1_128k", op="evict", cache="bf16", B=1, Hkv=8,
             D=128, S=131072, lo=131072, hi=131072, budget=16384, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.0e12 + w["flops"] / 1.5e15


def draw(rng):
    """One more case of the listed ranges (sizes spread over logarithms)."""
    op = rng.choice(["append", "attention", "attention", "weights", "evict"])
    cap = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        D = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 3, 4, 8, 8])
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 131072)
        lo = rng.randint(hi // 2, hi)
        if op == "append":
            n = _log_int(rng, 1, 8192)
            c = dict(op=op, B=B, n=n, Hkv=Hkv, D=D, S=hi + n + rng.randint(0, 9),
                     lo=lo, hi=hi)
        elif op == "evict":
            budget = _log_int(rng, 1, hi)
            c = dict(op=op, cache=rng.choice(["kv4", "bf16"]), B=B, Hkv=Hkv,
                     D=D, S=hi + rng.randint(0, 9), lo=lo, hi=hi,
                     budget=budget, recent=rng.randint(0, budget))
        else:
            N = rng.choice([1, 1, _log_int(rng, 1, 64)])
            G = rng.choice([1, 2, 4, 4, 7, 8])
            c = dict(op=op, B=B, N=N, Hq=G * Hkv, Hkv=Hkv, D=D,
                     S=hi + N + rng.randint(0, 9), lo=lo, hi=hi)
            if op == "weights":
                c["cache"] = rng.choice(["kv4", "bf16"])
        # the cache (and a weight row of every head) stays within 3 GB
        rows = c["B"] * c["Hkv"] * c["S"]
        scores = c["Hkv"] * c.get("N", 1) * (c.get("Hq", 1) // Hkv) * c["S"]
        if (_cost(c) <= cap and rows * (c["D"] * 4 + 8) < 10e9
                and scores * 4 < 4e9):
            return c


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written
    once."""
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    row4 = D // 2 + D // BLOCK          # one position's codes and scales
    pre = _prefix_values(case)
    if case["op"] == "append":
        el = B * case["n"] * Hkv
        # k and v read, codes and scales written, their values written back
        return {"bytes": 2 * el * (2 * D + row4 + 2 * D),
                "flops": 2 * el * D * 4}
    if case["op"] == "evict":
        row = 2 * row4 if case["cache"] == "kv4" else 4 * D
        kept = sum(min(x, case["budget"]) for x in pre) * Hkv
        return {"bytes": sum(pre) * Hkv * 4 + kept * (2 * row + 4 + 4),
                "flops": sum(pre) * Hkv * 4}
    N, Hq = case["N"], case["Hq"]
    if case["op"] == "attention":
        keys = sum(x + N for x in pre) * Hkv
        G = Hq // Hkv
        return {"bytes": keys * 2 * row4 + B * N * Hq * (4 * D + 4),
                "flops": 4 * keys * N * G * D}
    rows = min(N, PATH) * (Hq // Hkv)
    keys = sum(x + min(N, PATH) for x in pre) * Hkv
    krow = row4 if case["cache"] == "kv4" else 2 * D
    return {"bytes": keys * (krow + 8) + B * min(N, PATH) * Hq * (2 * D + 4),
            "flops": 2 * keys * rows * D}


PATH = 6                        # longest accepted path of the drawn trees


# ------------------------------------------------------------------ inputs
def _prefix_values(case):
    """The sequences' lengths: evenly spread over [lo, hi] (the seed only
    permutes them, so every seed means the same work)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    return [lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _trees(B, N, seed):
    """Random trees (parents among the six nodes before), their mask rows as
    64-bit words and a random root path of each."""
    import random
    rnd = random.Random(seed * 7919 + 13)
    bits, paths, lens = [], [], []
    for _ in range(B):
        parent = [-1 if j == 0 or rnd.random() < 0.15
                  else rnd.randint(max(0, j - 6), j - 1) for j in range(N)]
        word = []
        for j in range(N):
            word.append((word[parent[j]] if parent[j] >= 0 else 0) | (1 << j))
        bits.append([w - (1 << 64) if w >> 63 else w for w in word])
        path = [0]
        while len(path) < PATH:
            kids = [j for j in range(N) if parent[j] == path[-1]]
            if not kids:
                break
            path.append(rnd.choice(kids))
        lens.append(len(path))
        paths.append(path + [-1] * (N - len(path)))
    t = lambda x, dt: torch.tensor(x, dtype=dt, device=DEV)
    return t(bits, torch.int64), t(paths, torch.int32), t(lens, torch.int32)


def _keys(g, shape, D):
    """Key-like values: channels of unequal size, a few of them large."""
    amp = torch.exp(0.4 * torch.randn(D, generator=g, device=DEV))
    amp[torch.randperm(D, generator=g, device=DEV)[:max(1, D // 32)]] *= 3.0
    return torch.randn(*shape, D, generator=g, device=DEV) * amp


K_UNIT, V_UNIT = 1.0, 0.125


def _make_cache(case, pre, g, new):
    """A 4-bit (or bfloat16) cache whose first pre[b] + new positions hold
    keys and values; what lies behind them is left over from other use."""
    B, Hkv, S, D = case["B"], case["Hkv"], case["S"], case["D"]
    if case.get("cache", "kv4") == "bf16":
        k = torch.empty(B, Hkv, S, D, dtype=torch.bfloat16, device=DEV)
        v = torch.empty_like(k)
        for b in range(B):
            k[b] = _keys(g, (Hkv, S), D)
            v[b] = torch.randn(Hkv, S, D, generator=g, device=DEV) * 0.5
        return k, v
    u8 = lambda *s: torch.full(s, 0x7F, dtype=torch.uint8, device=DEV)
    kc, vc = u8(B, Hkv, S, D // 2), u8(B, Hkv, S, D // 2)
    ks, vs = u8(B, Hkv, S, D // BLOCK), u8(B, Hkv, S, D // BLOCK)
    for b in range(B):
        L = min(S, pre[b] + new)
        x = _keys(g, (Hkv, L), D).bfloat16()
        kc[b, :, :L], ks[b, :, :L] = _quantise(x, K_UNIT)
        x = (torch.randn(Hkv, L, D, generator=g, device=DEV) * 0.5).bfloat16()
        vc[b, :, :L], vs[b, :, :L] = _quantise(x, V_UNIT)
    return kc, ks, vc, vs


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, Hkv, S, D = case["B"], case["Hkv"], case["S"], case["D"]
    vals = _prefix_values(case)
    perm = torch.randperm(B, generator=g, device=DEV).tolist()
    pre = [vals[i] for i in perm]
    st = {"case": case, "pre": pre,
          "prefix": torch.tensor(pre, dtype=torch.int32, device=DEV)}
    if case["op"] == "append":
        n = case["n"]
        st["k"] = _keys(g, (B, n, Hkv), D).bfloat16()
        st["v"] = (torch.randn(B, n, Hkv, D, generator=g, device=DEV)
                   * 0.5).bfloat16()
        z = lambda w: torch.zeros(B, Hkv, S, w, dtype=torch.uint8, device=DEV)
        st["cache"] = (z(D // 2), z(D // BLOCK), z(D // 2), z(D // BLOCK))
        return st
    if case["op"] == "evict":
        st["cache"] = _make_cache(case, pre, g, 0)
        w = torch.exp(2.0 * torch.randn(B, Hkv, S, generator=g, device=DEV))
        # positions no row ever looked at: exact zeros, decided by index
        w[torch.rand(B, Hkv, S, generator=g, device=DEV) < 0.2] = 0.0
        st["weights"] = w
        k = case["budget"]
        st["planes_out"] = tuple(
            torch.zeros(B, Hkv, k, p.shape[-1], dtype=p.dtype, device=DEV)
            for p in st["cache"])
        st["weights_out"] = torch.zeros(B, Hkv, k, device=DEV)
        return st
    N, Hq = case["N"], case["Hq"]
    st["q"] = (torch.randn(B, N, Hq, D, generator=g, device=DEV)
               * 1.2).bfloat16()
    st["bits"], st["path"], st["path_len"] = _trees(B, N, seed)
    st["cache"] = _make_cache(case, pre, g, N)
    st["scale"] = D ** -0.5
    if case["op"] == "weights":
        # after a commit the accepted drafts follow the prefix; the rows'
        # normalisers are over the prefix and the path up to themselves
        st["lse"] = torch.zeros(B, N, Hq, device=DEV)
        lens = st["path_len"].tolist()
        for b in range(B):
            L = pre[b] + lens[b]
            kf = _key_values(st, b, L, torch.float32)
            rows = st["path"][b, :lens[b]].long()
            for t in range(lens[b]):
                q = st["q"][b, rows[t]].float().reshape(Hkv, -1, D)
                s = q @ kf[:, :pre[b] + t + 1].transpose(1, 2) * st["scale"]
                st["lse"][b, rows[t]] = (torch.logsumexp(s, -1)
                                         * LOG2E).reshape(Hq)
        st["weights"] = torch.rand(B, Hkv, S, generator=g, device=DEV) * 3.0
        st["out"] = torch.zeros(B, Hkv, S, device=DEV)
    return st


# -------------------------------------------------------- plain forms (f32)
def _quantise(x, unit):
    """x [..., D] -> (codes [..., D/2], scales [..., D/16]) uint8."""
    lead, D = x.shape[:-1], x.shape[-1]
    xb = x.float().reshape(*lead, D // BLOCK, BLOCK)
    a = xb.abs()
    s = (a.amax(-1) / (6.0 * unit)).clamp(min=2.0 ** -9, max=448.0)
    s = s.to(torch.float8_e4m3fn)
    r = a / (s.float() * unit).unsqueeze(-1)
    code = ((r > 0.25).to(torch.uint8) + (r >= 0.75) + (r > 1.25)
            + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5.0))
    code = code.to(torch.uint8) | (torch.signbit(xb).to(torch.uint8) << 3)
    code = code.reshape(*lead, D)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _values(codes, scales, unit):
    """The float32 values that codes and scales stand for."""
    lut = torch.tensor(CODE_VALUES, device=codes.device)
    lut = torch.cat([lut, -lut])
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    s = scales.view(torch.float8_e4m3fn).float() * unit
    return lut[c] * s.repeat_interleave(BLOCK, -1)


def _key_values(st, b, L, dtype):
    c = st["cache"]
    if len(c) == 2:
        return c[0][b, :, :L].to(dtype)
    return _values(c[0][b, :, :L], c[1][b, :, :L], K_UNIT).to(dtype)


def _plain_append(st):
    n, pre = st["case"]["n"], st["pre"]
    kc, ks, vc, vs = st["cache"]
    k4, k4s = _quantise(st["k"].transpose(1, 2), K_UNIT)
    v4, v4s = _quantise(st["v"].transpose(1, 2), V_UNIT)
    for b, p in enumerate(pre):
        kc[b, :, p:p + n], ks[b, :, p:p + n] = k4[b], k4s[b]
        vc[b, :, p:p + n], vs[b, :, p:p + n] = v4[b], v4s[b]
    rd = lambda c, s, u: torch.stack(
        [_values(c[b, :, p:p + n], s[b, :, p:p + n], u).transpose(0, 1)
         for b, p in enumerate(pre)]).bfloat16()
    return rd(kc, ks, K_UNIT), rd(vc, vs, V_UNIT)


def _visible(bits_b, P, N):
    sel = torch.arange(N, device=DEV)
    tree = ((bits_b.unsqueeze(1) >> sel) & 1).bool()
    return torch.cat([torch.ones(N, P, dtype=torch.bool, device=DEV), tree], 1)


def _plain_attention(st):
    c = st["case"]
    N, Hq, Hkv, D = c["N"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    outs, lses = [], []
    for b, P in enumerate(st["pre"]):
        L = P + N
        k = _key_values(st, b, L, torch.float32)
        v = _values(st["cache"][2][b, :, :L], st["cache"][3][b, :, :L], V_UNIT)
        q = st["q"][b].float().reshape(N, Hkv, G, D).permute(1, 0, 2, 3)
        s = q.reshape(Hkv, N * G, D) @ k.transpose(1, 2) * st["scale"]
        vis = _visible(st["bits"][b], P, N).repeat_interleave(G, 0)
        s = s.masked_fill(~vis, float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
        l = p.sum(-1, keepdim=True)
        o = torch.where(l > 0, (p @ v) / l, 0.0)
        lse = (m + torch.log(l)) * LOG2E
        outs.append(o.reshape(Hkv, N, G, D).permute(1, 0, 2, 3)
                    .reshape(N, Hq, D).bfloat16())
        lses.append(lse.reshape(Hkv, N, G).transpose(0, 1).reshape(N, Hq))
    return torch.stack(outs), torch.stack(lses)


def _plain_weights(st):
    c = st["case"]
    Hq, Hkv, D, N = c["Hq"], c["Hkv"], c["D"], c["N"]
    G, out = Hq // Hkv, st["out"]
    t = torch.arange(N, device=DEV)
    pos = torch.arange(c["S"], device=DEV)
    lens = st["path_len"].tolist()
    for b, P in enumerate(st["pre"]):
        n, L = lens[b], P + lens[b]
        k = _key_values(st, b, L, torch.float32)
        rows = st["path"][b, :n].long()
        q = st["q"][b, rows].float().reshape(n, Hkv, G, D).permute(1, 0, 2, 3)
        s = q.reshape(Hkv, n * G, D) @ k.transpose(1, 2) * (st["scale"] * LOG2E)
        lse = st["lse"][b, rows].reshape(n, Hkv, G).transpose(0, 1)
        w = torch.exp2(s - lse.reshape(Hkv, n * G, 1))
        seen = (pos[:L] <= P + t[:n, None]).repeat_interleave(G, 0)
        w = (w * seen).sum(1)
        out[b, :, :P] = st["weights"][b, :, :P] + w[:, :P]
        out[b, :, P:L] = w[:, P:]
    return out


def _plain_evict(st):
    c = st["case"]
    Hkv, k, r = c["Hkv"], c["budget"], c["recent"]
    kept = torch.full((c["B"], Hkv, k), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(st["pre"]):
        m = min(n, k)
        if n <= k:
            idx = torch.arange(n, device=DEV).expand(Hkv, n)
        else:
            w = st["weights"][b, :, :n - r]
            top = torch.sort(w, dim=-1, descending=True, stable=True)[1]
            old = torch.sort(top[:, :k - r], dim=-1)[0]
            new = torch.arange(n - r, n, device=DEV).expand(Hkv, r)
            idx = torch.cat([old, new], 1)
        kept[b, :, :m] = idx.int()
        st["weights_out"][b, :, :m] = st["weights"][b].gather(1, idx)
        for src, dst in zip(st["cache"], st["planes_out"]):
            dst[b, :, :m] = src[b].gather(
                1, idx.unsqueeze(-1).expand(-1, -1, src.shape[-1]))
    new_len = torch.clamp(st["prefix"], max=k)
    return (kept, new_len, st["weights_out"]) + st["planes_out"]


# ------------------------------------------------------ the library's calls
def _own(st):
    from speculative_decoding_verification_tree_gb300 import api
    c, op = st["case"], st["case"]["op"]
    if op == "append":
        cache = api.KV4Cache(*st["cache"])
        api.spec_kv4_append(st["k"], st["v"], st["prefix"], cache,
                            k_unit=K_UNIT, v_unit=V_UNIT)
        return api.spec_kv4_read(cache, st["prefix"], c["n"], k_unit=K_UNIT,
                                 v_unit=V_UNIT)
    if op == "attention":
        return api.spec_tree_attention_kv4(
            st["q"], api.KV4Cache(*st["cache"]), st["prefix"], st["bits"],
            scale=st["scale"], k_unit=K_UNIT, v_unit=V_UNIT, lse=True)
    if op == "weights":
        k = st["cache"][0] if c["cache"] == "bf16" else st["cache"][:2]
        return api.spec_kv_weights(
            st["q"], k, st["lse"], st["prefix"], st["path_len"], st["path"],
            scale=st["scale"], k_unit=K_UNIT if c["cache"] == "kv4" else 1.0,
            weights=st["weights"], out=st["out"])
    kept, new_len = api.spec_kv_evict(
        st["weights"], st["prefix"], st["cache"], budget=c["budget"],
        recent=c["recent"], weights_out=st["weights_out"],
        planes_out=st["planes_out"])
    return (kept, new_len, st["weights_out"]) + st["planes_out"]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attention": _plain_attention,
            "weights": _plain_weights,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ---------------------------------------------------- the definition, 64 bit
def _e4m3_table():
    """The 127 finite non-negative e4m3 values, in code order."""
    t = [m * 2.0 ** -9 for m in range(8)]
    t += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return t[:127]


def _nearest(x, table):
    """Index of the table value nearest to x >= 0 (ties: the even index)."""
    tab = torch.tensor(table, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(tab, x).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = x - tab[lo], tab[hi] - x
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    return torch.where(take_lo, lo, hi), tab


def _exact_append(x, unit):
    x = x.double()
    a = x.unflatten(-1, (-1, BLOCK))
    i, tab = _nearest(a.abs().amax(-1) / 6.0 / unit, _e4m3_table())
    s = tab[i.clamp(min=1)].unsqueeze(-1) * unit
    j, codes = _nearest(a.abs() / s, CODE_VALUES)
    return (torch.sign(a) * codes[j] * s).flatten(-2)


def _decode64(codes, scales, unit):
    """Values from the bit fields: (-1)^s 2^e (1 + m/2) and e4m3 likewise."""
    def field(c, mbits, bias):
        e, m = c >> mbits, (c & ((1 << mbits) - 1)).double() / (1 << mbits)
        return torch.where(e > 0, (1 + m) * torch.exp2((e - bias).double()),
                           m * 2.0 ** (1 - bias))
    c = codes.int()
    c = torch.stack([c % 16, c // 16], -1).flatten(-2)
    val = field(c & 7, 1, 1) * (1 - 2 * (c >> 3)).double()
    s = scales.int()
    sc = field(s & 127, 3, 7) * (1 - 2 * (s >> 7)).double() * unit
    return (val.unflatten(-1, (-1, BLOCK)) * sc.unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return (_exact_append(st["k"], K_UNIT), _exact_append(st["v"], V_UNIT))
    if op == "evict":
        kept, new_len, w = _exact_evict(st)
        return (kept, new_len, w) + (None,) * len(st["planes_out"])
    N, Hq, Hkv = case["N"], case["Hq"], case["Hkv"]
    G, c = Hq // Hkv, st["cache"]
    D = case["D"]
    if op == "attention":
        out = torch.zeros(case["B"], N, Hq, D, dtype=torch.float64, device=DEV)
        lse = torch.zeros(case["B"], N, Hq, dtype=torch.float64, device=DEV)
    else:
        out = torch.zeros(case["B"], Hkv, case["S"], dtype=torch.float64,
                          device=DEV)
    lens = st["path_len"].tolist()
    paths, words = st["path"].tolist(), st["bits"].tolist()
    for b, P in enumerate(st["pre"]):
        new = N if op == "attention" else lens[b]
        for h in range(Hkv):
            if len(c) == 2:
                k = c[0][b, h, :P + new].double()
            else:
                k = _decode64(c[0][b, h, :P + new], c[1][b, h, :P + new],
                              K_UNIT)
            heads = slice(h * G, h * G + G)
            if op == "weights":
                acc = torch.zeros(P + new, dtype=torch.float64, device=DEV)
                for t in range(new):
                    i = paths[b][t]
                    z = (k[:P + t + 1] @ st["q"][b, i, heads].double().T
                         * st["scale"])
                    acc[:P + t + 1] += torch.exp(
                        z - st["lse"][b, i, heads].double() * math.log(2)
                    ).sum(1)
                out[b, h, :P + new] = acc
                out[b, h, :P] += st["weights"][b, h, :P].double()
                continue
            v = _decode64(c[2][b, h, :P + new], c[3][b, h, :P + new], V_UNIT)
            hide = torch.tensor([[not (w >> j) & 1 for w in words[b]]
                                 for j in range(N)], device=DEV)
            qd = st["q"][b, :, heads].double()              # [N, G, D]
            z = torch.einsum("sd,ngd->ngs", k, qd) * st["scale"]
            z[:, :, P:] = z[:, :, P:].masked_fill(hide.T.unsqueeze(1),
                                                  -math.inf)
            norm = torch.logsumexp(z, -1)
            out[b, :, heads] = torch.exp(z - norm.unsqueeze(-1)) @ v
            lse[b, :, heads] = norm / math.log(2)
    return (out, lse) if op == "attention" else out


def _exact_evict(st):
    """Rank every position by counting the ones that beat it (heavier, or
    equal and earlier), on the host."""
    import numpy as np
    c, w = st["case"], st["weights"].double().cpu().numpy()
    k, r = c["budget"], c["recent"]
    kept = np.full((c["B"], c["Hkv"], k), -1, dtype=np.int32)
    out = np.zeros((c["B"], c["Hkv"], k))
    for b, n in enumerate(st["pre"]):
        for h in range(c["Hkv"]):
            if n <= k:
                idx = np.arange(n)
            else:
                order = np.lexsort((np.arange(n - r), -w[b, h, :n - r]))
                idx = np.sort(np.concatenate([order[:k - r],
                                              np.arange(n - r, n)]))
            kept[b, h, :len(idx)] = idx
            out[b, h, :len(idx)] = w[b, h, idx]
    return (torch.from_numpy(kept).to(DEV),
            torch.tensor([min(n, k) for n in st["pre"]], dtype=torch.int32,
                         device=DEV), torch.from_numpy(out).to(DEV))
