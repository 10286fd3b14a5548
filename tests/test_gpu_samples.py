"""Several samples of one prompt: the operators as a loop uses them together.

The prompt is read once (spec_prompt_attention), its keys and values become the
shared prefix; every step drafts a tree per sample, attends over prefix, own
keys and tree (spec_tree_attention_shared), verifies through the LM head, rates
the emitted tokens (spec_token_logprobs) and commits the accepted entries.
Checked: the shared attention of chains equals the prompt attention over the
same tokens written out (both within their tolerance of each other), that of
trees the oracle; the ratings equal the oracle's on the same logits; and the
gradient of the ratings the oracle's.
"""

import numpy as np
import pytest
import torch

from oracle import logprobs as lp_oracle
from oracle import shared as oracle
from oracle.tree import tree_mask
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
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


B, HQ, HKV, D, V, H = 5, 8, 2, 128, 1000, 8 * 128
P = 300                                         # the prompt's tokens


class Layer:
    """Random keys, values and queries per (sequence, position, token id)."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def draw(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").bfloat16()


def prefix_of(k):
    """Packed [T, Hkv, D] as the one-prefix cache [1, Hkv, T, D]."""
    return k.transpose(0, 1).unsqueeze(0).contiguous()


def test_chains_equal_the_prompt_written_out():
    a, ly = api(), Layer(0)
    own = [0, 3, 17, 130, 64]
    N = 6
    q, k, v = (ly.draw(P, h, D) for h in (HQ, HKV, HKV))
    S = max(own) + N
    kc, vc = ly.draw(B, HKV, S, D), ly.draw(B, HKV, S, D)
    qn = ly.draw(B, N, HQ, D)
    par = np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1))
    _, bits = a.spec_tree_mask(i32(par), bits=True, mask=False)
    out, lse = a.spec_tree_attention_shared(
        qn, prefix_of(k), prefix_of(v), i32([P]), i32([0, B]), kc, vc,
        i32(own), bits, lse=True)
    # every sample as a prompt of its own: prompt, own tokens, drafts
    seqs, starts = [], [0]
    for b in range(B):
        L = own[b] + N
        qs = torch.cat([q, ly.draw(own[b], HQ, D), qn[b]])
        ks = torch.cat([k, kc[b, :, :L].transpose(0, 1)])
        vs = torch.cat([v, vc[b, :, :L].transpose(0, 1)])
        seqs.append((qs, ks, vs))
        starts.append(starts[-1] + P + L)
    packed = [torch.cat(x).contiguous() for x in zip(*seqs)]
    o2, l2 = a.spec_prompt_attention(*packed, i32(starts), lse=True)
    for b in range(B):
        r = slice(starts[b + 1] - N, starts[b + 1])
        # both within 2^-8 (|o| + A) and float32 steps of the exact value, with
        # |o| <= A <= max |v|
        amax = float(v.float().abs().max().clamp(min=vc.float().abs().max()))
        assert (out[b].float() - o2[r].float()).abs().max() <= 4.2 * 2 ** -8 * amax
        assert (lse[b] - l2[r]).abs().max() <= 2 ** -10
    # and the prompt's own rows do not depend on what follows
    o1, l1 = a.spec_prompt_attention(q, k, v, i32([0, P]), lse=True)
    for b in range(B):
        r = slice(starts[b], starts[b] + P)
        assert torch.equal(o2[r], o1) and torch.equal(l2[r], l1)


def test_steps_of_a_sampling_loop():
    a, ly = api(), Layer(1)
    rng = np.random.default_rng(1)
    N, S = 9, 80
    q, k, v = (ly.draw(P, h, D) for h in (HQ, HKV, HKV))
    a.spec_prompt_attention(q, k, v, i32([0, P]))
    kp, vp = prefix_of(k), prefix_of(v)
    kc, vc = (torch.zeros(B, HKV, S, D, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    w_vocab = (ly.draw(V, H).float() * (2 / H ** 0.5)).bfloat16()
    length = i32([0] * B)
    row = D * 2
    layout = (1, HKV, HKV * S * row, 0, S * row, row)
    for step in range(3):
        pre = length.tolist()
        par = random_parent(rng, B, N)
        _, bits = a.spec_tree_mask(i32(par), bits=True, mask=False)
        for b in range(B):                      # the drafts' keys and values
            kc[b, :, pre[b]:pre[b] + N] = ly.draw(HKV, N, D)
            vc[b, :, pre[b]:pre[b] + N] = ly.draw(HKV, N, D)
        qn = ly.draw(B, N, HQ, D)
        args = (qn, kp, vp, i32([P]), i32([0, B]), kc, vc, length, bits)
        out, lse = a.spec_tree_attention_shared(*args, lse=True)
        want, l, mag, sm = oracle.tree_attention_shared(
            np64(qn), np64(kp), np64(vp), [P], [0, B], np64(kc), np64(vc), pre,
            tree_mask(par)[1], D ** -0.5)
        n = P + max(pre) + N
        tol = (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -16 * sm[..., None]
               + (n / 16 + 400) * 2.0 ** -23) * mag)
        assert (np.abs(np64(out) - want) <= tol).all()
        # target logits at the root (the last emitted token) and at every node
        hidden = torch.cat([ly.draw(B, 1, H), out.reshape(B, N, H)], 1)
        logits, _ = a.spec_lm_head(hidden.contiguous(), w_vocab)
        tokens = torch.from_numpy(np.stack([
            rng.choice(V, N, replace=False) for _ in range(B)])).int().cuda()
        for b in range(B):                      # probable drafts under the root
            tokens[b, 0] = logits[b, 0].float().argmax().int()
        draft = ly.draw(B, N + 1, V).float()
        qrow = i32(np.tile(np.arange(N + 1), (B, 1)))
        path_len, path, emitted, _ = a.spec_verify_tree(
            logits, draft, qrow, tokens, i32(par), temperature=1.0,
            seed=step)
        # the emitted tokens under the rows that decided them
        at = torch.cat([torch.zeros(B, 1, dtype=torch.int32, device="cuda"),
                        path + 1], 1)
        at[:, 1:][path < 0] = -1
        rows = torch.where(at >= 0, at + i32(np.arange(B) * (N + 1))[:, None],
                           at)
        r = a.spec_token_logprobs(logits, emitted, rows=rows.contiguous(),
                                  top=4, entropy=True)
        lens = path_len.tolist()
        z = np64(logits)
        for b in range(B):
            m = lens[b] + 1                     # tokens emitted by sequence b
            pick = [0] + (path[b, :lens[b]] + 1).tolist()
            lp, nz, ent, ids, tl = lp_oracle.token_logprobs(
                z[b, pick], emitted[b, :m].cpu().numpy()[:, None], 1.0, 4)
            assert np.abs(np64(r.logprob[b, :m]) - lp[:, 0]).max() <= 2 ** -14
            assert np.abs(np64(r.entropy[b, :m]) - ent).max() <= 2 ** -12
            assert np.array_equal(r.top_ids[b, :m].cpu().numpy(), ids)
            assert (r.logprob[b, m:] == 0).all()
            assert (r.top_ids[b, m:] == -1).all()
        # the gradient of the sum of the root tokens' log probabilities
        root = logits[:, 0]
        f = a.spec_token_logprobs(root, emitted[:, 0].contiguous())
        g = a.spec_token_logprobs_grad(root, emitted[:, 0].contiguous(), f.lse,
                                       torch.ones(B, device="cuda"))
        want = lp_oracle.grad(z[:, 0], emitted[:, :1].cpu().numpy(),
                              np.ones((B, 1)))
        assert (np.abs(np64(g) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5).all()
        for plane in (kc, vc):
            new = a.spec_kv_commit(plane, length, path_len, path, row_bytes=row,
                                   N=N, layout=layout)
        assert new.tolist() == [p + n for p, n in zip(pre, lens)]
        length = new
