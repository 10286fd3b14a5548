"""Cases and plain forms of the operators around several answers to one prompt.

Four operators of a loop that reads a prompt, continues it many times with
tree verification and rates the answers:

  prompt    causal attention over whole prompts, packed one after another,
            with grouped heads: the pass that fills the cache
  shared    tree / single-token attention of sequences that share a long
            prefix and have keys of their own behind it
  logprobs  log probabilities of given tokens, the rows' entropy and the most
            probable alternatives, from logits
  grad      the gradient of those log probabilities and entropies with
            respect to the logits

`own` selects what `run` calls: the plain forms below (elementary torch
operations in float32) or the library's entry points.
"""

import math

import torch

own = False

LOG2E = 1.4426950408889634
DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one short prompt of a chat: the time to the first token
        dict(name="prompt_b1_1000", op="prompt", B=1, lo=1000, hi=1000, Hq=32,
             Hkv=8, D=128, fused=True),
        # a batch of prompts admitted together, ragged
        dict(name="prompt_b16_ragged", op="prompt", B=16, lo=37, hi=4095,
             Hq=32, Hkv=8, D=128, fused=True),
        # one long document
        dict(name="prompt_b1_16k", op="prompt", B=1, lo=16384, hi=16384,
             Hq=32, Hkv=8, D=128, fused=False),
        # a small draft model's odd sizes: 7 query heads per key/value head,
        # head dim 64, a one-token prompt among them
        dict(name="prompt_b7_odd_d64", op="prompt", B=7, lo=1, hi=2501, Hq=14,
             Hkv=2, D=64, fused=False),
        # 32 samples of one long prompt, a token at a time
        dict(name="shared_decode_b32_32k", op="shared", B=32, N=1, groups=1,
             Hq=32, Hkv=8, D=128, slo=32768, shi=32768, lo=1, hi=1000, S=1024),
        # verification of 60-node trees of 16 samples behind a prompt of 8 K
        dict(name="shared_tree_b16_8k", op="shared", B=16, N=60, groups=1,
             Hq=32, Hkv=8, D=128, slo=8192, shi=8192, lo=100, hi=1000,
             S=1100),
        # five prompts with a few samples each, odd sizes of a small model
        dict(name="shared_g5_odd_d64", op="shared", B=13, N=7, groups=5,
             Hq=14, Hkv=2, D=64, slo=333, shi=5003, lo=0, hi=701, S=711),
        # one step of a single chain: the emitted token's log probability and
        # five alternatives; latency is everything
        dict(name="logprobs_b1", op="logprobs", M=1, V=32000, n=1, top=5,
             dtype="f32", T=1.0, pick=False, entropy=False, pad=0),
        # the tokens a step with 60-node trees emitted for 32 sequences, their
        # rows picked out of the target's logits, twenty alternatives each
        dict(name="logprobs_tree_b32", op="logprobs", M=224, V=128256, n=1,
             top=20, dtype="bf16", T=1.0, pick=True, entropy=True, pad=0),
        # rating 8192 tokens of finished answers under the target model
        dict(name="logprobs_8k", op="logprobs", M=8192, V=128256, n=1, top=0,
             dtype="bf16", T=1.0, pick=False, entropy=True, pad=0),
        # the same rows' gradient when a draft model is trained on 4096 tokens
        dict(name="grad_4k", op="grad", M=4096, V=128256, n=1, dtype="bf16",
             T=1.0, entropy=True, pad=0),
        # an odd vocabulary inside padded rows, three given tokens a row
        dict(name="grad_odd_f32", op="grad", M=777, V=50257, n=3,
             dtype="f32", T=0.7, entropy=False, pad=47),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.0e12 + w["flops"] / 1.5e15


def draw(rng):
    """One more case of the listed ranges (sizes spread over logarithms)."""
    op = rng.choice(["prompt", "prompt", "shared", "shared", "logprobs",
                     "grad"])
    cap = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        D = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 3, 4, 8, 8])
        G = rng.choice([1, 2, 4, 4, 5, 7, 8])
        if op == "prompt":
            hi = _log_int(rng, 1, 16384)
            c = dict(op=op, B=_log_int(rng, 1, 64), lo=rng.randint(1, hi),
                     hi=hi, Hq=G * Hkv, Hkv=Hkv, D=D,
                     fused=rng.random() < 0.5)
            fits = _total(c) <= 40000
        elif op == "shared":
            N = rng.choice([1, 1, _log_int(rng, 1, 64)])
            B = _log_int(rng, 1, 64)
            shi, hi = _log_int(rng, 1, 65536), _log_int(rng, 1, 2048)
            c = dict(op=op, B=B, N=N, groups=rng.choice([1, 1, min(B, 3)]),
                     Hq=G * Hkv, Hkv=Hkv, D=D, slo=rng.randint(shi // 2, shi),
                     shi=shi, lo=rng.randint(0, hi), hi=hi,
                     S=hi + N + rng.randint(0, 9))
            # one sequence's scores in 32 bits stay within 4 GB
            fits = (shi + hi + N) * N * G * Hkv < 1e9
        else:
            V = _log_int(rng, 1000, 160000)
            V += (-V) % 8 if rng.random() < 0.5 else 0
            c = dict(op=op, M=_log_int(rng, 1, 8192), V=V,
                     n=rng.choice([1, 1, 3, 10]),
                     dtype=rng.choice(["bf16", "bf16", "f32"]),
                     T=rng.choice([1.0, 1.0, 0.6, 1.3]),
                     entropy=rng.random() < 0.5,
                     pad=rng.choice([0, 0, 8, 47]))
            if op == "logprobs":
                c["top"] = rng.choice([0, 1, 5, 20])
                c["pick"] = rng.random() < 0.3
                # alternatives are sorted in the plain form
                fits = c["top"] == 0 or c["M"] * V < 1 << 28
            else:
                fits = True
        if fits and _cost(c) <= cap:
            return c


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written
    once."""
    if case["op"] in ("logprobs", "grad"):
        el = 4 if case["dtype"] == "f32" else 2
        M, V, n = case["M"], case["V"], case["n"]
        if case["op"] == "grad":
            return {"bytes": M * (2 * V * el + n * 8 + 12),
                    "flops": M * V * 6}
        return {"bytes": M * (V * el + n * 8 + 8 + case["top"] * 8),
                "flops": M * V * (7 if case["entropy"] else 5)}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "prompt":
        lens = _lengths(case["B"], case["lo"], case["hi"])
        pairs = sum(x * (x + 1) // 2 for x in lens)
        return {"bytes": sum(lens) * (2 * D * (2 * Hq + 2 * Hkv) + 4 * Hq),
                "flops": 4 * D * Hq * pairs}
    N = case["N"]
    own_keys = [x + N for x in _lengths(case["B"], case["lo"], case["hi"])]
    shared = _lengths(case["groups"], case["slo"], case["shi"])
    start = _group_start(case)
    keys = sum(own_keys) + sum(shared)
    seen = sum(own_keys) + sum(
        s * (start[g + 1] - start[g]) for g, s in enumerate(shared))
    return {"bytes": keys * Hkv * 4 * D + case["B"] * N * Hq * (4 * D + 4),
            "flops": 4 * D * Hq * N * seen}


# ------------------------------------------------------------------ inputs
def _lengths(B, lo, hi):
    """Lengths evenly spread over [lo, hi] (a seed only permutes them, so
    every seed means the same work)."""
    if B == 1:
        return [hi]
    return [lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _total(case):
    return sum(_lengths(case["B"], case["lo"], case["hi"]))


def _group_start(case):
    """Sequences per prefix, unequal where they do not divide."""
    n, B = case["groups"], case["B"]
    return [B * g // n for g in range(n)] + [B]


def _permuted(values, g):
    perm = torch.randperm(len(values), generator=g, device=DEV).tolist()
    return [values[i] for i in perm]


def _keys(g, shape, D):
    """Key-like values: channels of unequal size, a few of them large."""
    amp = torch.exp(0.4 * torch.randn(D, generator=g, device=DEV))
    amp[torch.randperm(D, generator=g, device=DEV)[:max(1, D // 32)]] *= 3.0
    return (torch.randn(*shape, D, generator=g, device=DEV) * amp).bfloat16()


def _normal(g, shape, std):
    return (torch.randn(*shape, generator=g, device=DEV) * std).bfloat16()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tree_words(B, N, seed):
    """Random trees (parents among the six nodes before) as mask rows of 64
    bits."""
    import random
    rnd = random.Random(seed * 7919 + 13)
    out = []
    for _ in range(B):
        word = []
        for j in range(N):
            p = (-1 if j == 0 or rnd.random() < 0.15
                 else rnd.randint(max(0, j - 6), j - 1))
            word.append((word[p] if p >= 0 else 0) | (1 << j))
        out.append([w - (1 << 64) if w >> 63 else w for w in word])
    return torch.tensor(out, dtype=torch.int64, device=DEV)


def _logits(case, g, rows):
    """Logits of a target model (bell-shaped, std 2.5), a thirtieth of the
    vocabulary masked off, as a view into rows with padding behind."""
    V, dt = case["V"], torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    z = torch.empty(rows, V + case["pad"], dtype=dt, device=DEV)
    off = torch.rand(V, generator=g, device=DEV) < 1 / 30
    for i in range(0, rows, 256):
        m = min(256, rows - i)
        x = torch.randn(m, V + case["pad"], generator=g, device=DEV) * 2.5
        x[:, :V].masked_fill_(off, float("-inf"))
        z[i:i + m] = x
    return z[:, :V], off


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, st = case["op"], {"case": case}
    if op == "prompt":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        lens = _permuted(_lengths(case["B"], case["lo"], case["hi"]), g)
        T = sum(lens)
        q, k = _normal(g, (T, Hq, D), 1.2), _keys(g, (T, Hkv), D)
        v = _normal(g, (T, Hkv, D), 0.5)
        if case["fused"]:       # slices of one projection's output
            x = torch.cat([q, k, v], 1)
            q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        start = [0]
        for n in lens:
            start.append(start[-1] + n)
        st.update(q=q, k=k, v=v, starts=start, start=_i32(start),
                  scale=D ** -0.5)
        return st
    if op == "shared":
        Hq, Hkv, D, N = case["Hq"], case["Hkv"], case["D"], case["N"]
        B, S, n = case["B"], case["S"], case["groups"]
        slen = _permuted(_lengths(n, case["slo"], case["shi"]), g)
        pre = _permuted(_lengths(B, case["lo"], case["hi"]), g)
        Sp = max(slen) + 3
        st.update(
            slen=slen, pre=pre, starts=_group_start(case),
            shared_len=_i32(slen), prefix=_i32(pre),
            group=_i32(_group_start(case)),
            q=_normal(g, (B, N, Hq, D), 1.2), bits=_tree_words(B, N, seed),
            pk=_keys(g, (n, Hkv, Sp), D), pv=_normal(g, (n, Hkv, Sp, D), 0.5),
            k=_keys(g, (B, Hkv, S), D), v=_normal(g, (B, Hkv, S, D), 0.5),
            scale=D ** -0.5)
        return st
    M, V, n = case["M"], case["V"], case["n"]
    pick = case.get("pick", False)
    st["logits"], off = _logits(case, g, M * 3 if pick else M)
    if pick:
        rows = torch.randperm(M * 3, generator=g, device=DEV)[:M]
        st["rows"] = rows.sort()[0].int()
    # given tokens: probable ones mostly (the best of 64 places), a few
    # absent (-1, as the verifier pads)
    at = st["rows"].long() if pick else torch.arange(M, device=DEV)
    spot = torch.randint(V, (M, n, 64), generator=g, device=DEV)
    best = torch.stack([st["logits"][at[:, None], spot[:, :, i]].float()
                        for i in range(64)], -1).argmax(-1, keepdim=True)
    tok = spot.gather(-1, best).squeeze(-1)
    tok[off[tok]] = -1
    st["tokens"] = tok.int().contiguous()
    if op == "grad":
        st["g_logprob"] = torch.randn(M, n, generator=g, device=DEV) / M
        lse, H = _normalisers(st["logits"], case["T"], torch.float64)
        st["lse"] = (lse * LOG2E).float()
        if case["entropy"]:
            st["entropy"] = H.float()
            st["g_entropy"] = (torch.randn(M, generator=g, device=DEV)
                               * 0.1 / M)
    return st


# -------------------------------------------------------- plain forms (f32)
def _attend(q, k, v, scale, vis):
    """q [Hkv, R, D], k, v [Hkv, L, D], vis [R, L] or None -> o [Hkv, R, D],
    lse [Hkv, R] (natural)."""
    s = q @ k.transpose(1, 2) * scale
    if vis is not None:
        s = s.masked_fill(~vis, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, (p @ v) / l, 0.0)
    return o, (m + torch.log(l)).squeeze(-1)


def _plain_prompt(st):
    c = st["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    T = st["starts"][-1]
    out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(T, Hq, device=DEV)
    for a, z in zip(st["starts"], st["starts"][1:]):
        k = st["k"][a:z].float().transpose(0, 1)
        v = st["v"][a:z].float().transpose(0, 1)
        for i in range(a, z, 1024):
            e = min(i + 1024, z)
            q = st["q"][i:e].float().reshape(e - i, Hkv, G, D)
            q = q.permute(1, 0, 2, 3).reshape(Hkv, -1, D)
            pos = torch.arange(i - a, e - a, device=DEV).repeat_interleave(G)
            vis = torch.arange(e - a, device=DEV) <= pos[:, None]
            o, l = _attend(q, k[:, :e - a], v[:, :e - a], st["scale"], vis)
            out[i:e] = (o.reshape(Hkv, e - i, G, D).transpose(0, 1)
                        .reshape(e - i, Hq, D).bfloat16())
            lse[i:e] = (l.reshape(Hkv, e - i, G).transpose(0, 1)
                        .reshape(e - i, Hq) * LOG2E)
    return out, lse


def _plain_shared(st):
    c = st["case"]
    N, Hq, Hkv, D = c["N"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    out = torch.empty_like(st["q"])
    lse = torch.empty(c["B"], N, Hq, device=DEV)
    sel = torch.arange(N, device=DEV)
    for g, n in enumerate(st["slen"]):
        for b in range(st["starts"][g], st["starts"][g + 1]):
            L = st["pre"][b] + N
            k = torch.cat([st["pk"][g, :, :n], st["k"][b, :, :L]], 1).float()
            v = torch.cat([st["pv"][g, :, :n], st["v"][b, :, :L]], 1).float()
            tree = ((st["bits"][b].unsqueeze(1) >> sel) & 1).bool()
            vis = torch.cat([torch.ones(N, n + L - N, dtype=torch.bool,
                                        device=DEV), tree], 1)
            q = st["q"][b].float().reshape(N, Hkv, G, D).permute(1, 0, 2, 3)
            o, l = _attend(q.reshape(Hkv, N * G, D), k, v, st["scale"],
                           vis.repeat_interleave(G, 0))
            out[b] = (o.reshape(Hkv, N, G, D).transpose(0, 1)
                      .reshape(N, Hq, D).bfloat16())
            lse[b] = (l.reshape(Hkv, N, G).transpose(0, 1).reshape(N, Hq)
                      * LOG2E)
    return out, lse


def _normalisers(logits, T, dtype):
    """Natural log normaliser and entropy of every row, in `dtype`."""
    lse, ent = [], []
    for z in logits.split(512):
        z = z.to(dtype) / T
        m = z.amax(-1, keepdim=True)
        e = torch.exp(z - m)
        s = e.sum(-1, keepdim=True)
        lp = z - m - torch.log(s)
        p = e / s
        ent.append(-torch.where(p > 0, p * lp, 0.0).sum(-1))
        lse.append((m + torch.log(s)).squeeze(-1))
    return torch.cat(lse), torch.cat(ent)


def _given(z, lse, tokens):
    """Log probabilities of the given tokens (0 where there is none)."""
    lp = z.gather(-1, tokens.clamp(min=0).long()) - lse.unsqueeze(-1)
    return torch.where(tokens >= 0, lp, 0.0)


def _plain_logprobs(st):
    c = st["case"]
    outs = []
    for i in range(0, c["M"], 512):
        e = min(i + 512, c["M"])
        rows = st["rows"][i:e].long() if c["pick"] else slice(i, e)
        raw = st["logits"][rows].float()
        z = raw / c["T"]
        lse, ent = _normalisers(raw, c["T"], torch.float32)
        out = [_given(z, lse, st["tokens"][i:e]), lse * LOG2E]
        if c["entropy"]:
            out.append(ent)
        if c["top"]:
            ids = torch.sort(z, dim=-1, descending=True, stable=True)[1]
            ids = ids[:, :c["top"]]
            out += [ids.int(), z.gather(-1, ids) - lse.unsqueeze(-1)]
        outs.append(out)
    return tuple(torch.cat(x) for x in zip(*outs))


def _plain_grad(st):
    c = st["case"]
    out = []
    for i in range(0, c["M"], 512):
        r = slice(i, i + 512)
        lp = st["logits"][r].float() / c["T"] - (st["lse"][r] / LOG2E)[:, None]
        p, tok = torch.exp(lp), st["tokens"][r]
        gl = torch.where(tok >= 0, st["g_logprob"][r], 0.0)
        t = gl.sum(-1, keepdim=True)
        if c["entropy"]:
            t = t + (st["g_entropy"][r][:, None]
                     * (torch.where(p > 0, lp, 0.0) + st["entropy"][r][:, None]))
        d = -p * t
        d.scatter_add_(1, tok.clamp(min=0).long(), gl)
        out.append((d / c["T"]).to(st["logits"].dtype))
    return torch.cat(out)


# ------------------------------------------------------ the library's calls
def _own(st):
    from speculative_decoding_verification_tree_gb300 import api
    c, op = st["case"], st["case"]["op"]
    if op == "prompt":
        return api.spec_prompt_attention(st["q"], st["k"], st["v"],
                                         st["start"], scale=st["scale"],
                                         lse=True)
    if op == "shared":
        return api.spec_tree_attention_shared(
            st["q"], st["pk"], st["pv"], st["shared_len"], st["group"],
            st["k"], st["v"], st["prefix"], st["bits"], scale=st["scale"],
            lse=True)
    if op == "grad":
        return api.spec_token_logprobs_grad(
            st["logits"], st["tokens"], st["lse"], st["g_logprob"],
            temperature=c["T"], entropy=st.get("entropy"),
            g_entropy=st.get("g_entropy"))
    r = api.spec_token_logprobs(st["logits"], st["tokens"],
                                temperature=c["T"], top=c["top"],
                                entropy=c["entropy"], rows=st.get("rows"))
    return tuple(x for x in (r.logprob, r.lse, r.entropy, r.top_ids,
                             r.top_logprob) if x is not None)


def run(state):
    if own:
        return _own(state)
    return {"prompt": _plain_prompt, "shared": _plain_shared,
            "logprobs": _plain_logprobs,
            "grad": _plain_grad}[state["case"]["op"]](state)


# ---------------------------------------------------- the definition, 64 bit
def _exact_attention(q, k, v, scale, hidden):
    """One query head: q [R, D], k, v [L, D], hidden [R, L] (True = masked):
    outputs and base-2 normalisers by log-sum-exp."""
    z = torch.einsum("rd,ld->rl", q.double(), k.double()).mul_(scale)
    z.masked_fill_(hidden, -math.inf)
    norm = torch.logsumexp(z, -1)
    return (z.sub_(norm.unsqueeze(-1)).exp_() @ v.double(),
            norm / math.log(2))


def _exact_prompt(st):
    c = st["case"]
    G, T = c["Hq"] // c["Hkv"], st["starts"][-1]
    out = torch.empty(T, c["Hq"], c["D"], dtype=torch.float64, device=DEV)
    lse = torch.empty(T, c["Hq"], dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        a, z = st["starts"][b], st["starts"][b + 1]
        for i in range(a, z, 4096):
            e = min(i + 4096, z)
            hidden = torch.ones(e - i, e - a, dtype=torch.bool,
                                device=DEV).triu(i - a + 1)
            for h in range(c["Hq"]):
                out[i:e, h], lse[i:e, h] = _exact_attention(
                    st["q"][i:e, h], st["k"][a:e, h // G],
                    st["v"][a:e, h // G], st["scale"], hidden)
    return out, lse


def _exact_shared(st):
    c = st["case"]
    B, N, Hq, G = c["B"], c["N"], c["Hq"], c["Hq"] // c["Hkv"]
    out = torch.empty(B, N, Hq, c["D"], dtype=torch.float64, device=DEV)
    lse = torch.empty(B, N, Hq, dtype=torch.float64, device=DEV)
    words = st["bits"].tolist()
    for b in range(B):
        g = max(i for i in range(c["groups"]) if st["starts"][i] <= b)
        n, P = st["slen"][g], st["pre"][b]
        hidden = torch.zeros(N, n + P + N, dtype=torch.bool)
        hidden[:, n + P:] = torch.tensor(
            [[not (w >> j) & 1 for j in range(N)] for w in words[b]])
        hidden = hidden.to(DEV)
        for h in range(Hq):
            kv = [torch.cat([x[g, h // G, :n], y[b, h // G, :P + N]])
                  for x, y in ((st["pk"], st["k"]), (st["pv"], st["v"]))]
            out[b, :, h], lse[b, :, h] = _exact_attention(
                st["q"][b, :, h], *kv, st["scale"], hidden)
    return out, lse


def _exact_rows(case, st):
    """Outputs of the logits' operators, a few rows at a time."""
    n, T, V = case["n"], case["T"], case["V"]
    fields = []
    for i in range(0, case["M"], 128):
        m = min(128, case["M"] - i)
        at = st["rows"][i:i + m].long() if "rows" in st else torch.arange(
            i, i + m, device=DEV)
        raw = st["logits"].index_select(0, at)
        z = raw.double().div(T)
        given = st["tokens"][i:i + m].long()
        norm = torch.logsumexp(z, -1)
        if case["op"] == "grad":
            norm = st["lse"][i:i + m].double() * math.log(2)
        logp = z - norm.view(m, 1)
        p = logp.exp()
        if case["op"] == "grad":
            d = torch.zeros_like(z)
            for j in range(n):
                hot = torch.zeros_like(z)
                r = torch.nonzero(given[:, j] >= 0).view(-1)
                hot[r, given[r, j]] = 1.0
                w = st["g_logprob"][i:i + m, j].double()
                w = w.masked_fill(given[:, j] < 0, 0.0)
                d += w.view(m, 1) * (hot - p)
            if case["entropy"]:
                H = st["entropy"][i:i + m].double().view(m, 1)
                u = p * (logp.masked_fill(p == 0, 0.0) + H)
                d -= st["g_entropy"][i:i + m].double().view(m, 1) * u
            fields.append([d / T])
            continue
        lp = torch.zeros(m, n, dtype=torch.float64, device=DEV)
        for j in range(n):
            r = torch.nonzero(given[:, j] >= 0).view(-1)
            lp[r, j] = logp[r, given[r, j]]
        f = [lp, norm / math.log(2)]
        if case["entropy"]:
            f.append(torch.special.entr(p).sum(-1))
        if case["top"]:
            # order by value, then by place: both in one integer key
            bits = raw.float().view(torch.int32).long()
            rank = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
            key = rank * 2 ** 24 + (2 ** 24 - 1 - torch.arange(V, device=DEV))
            ids = torch.topk(key, case["top"], -1)[1]
            f += [ids.int(), logp.gather(1, ids)]
        fields.append(f)
    out = tuple(torch.cat(x) for x in zip(*fields))
    return out[0] if case["op"] == "grad" else out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(st)
    if case["op"] == "shared":
        return _exact_shared(st)
    return _exact_rows(case, st)
