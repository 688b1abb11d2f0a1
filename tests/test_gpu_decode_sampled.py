"""Sampled generation: pages from lengths, capped attention, filtered drafts and targets, verified and kept, step after step.

Every emitted token has to be one that the target's filter allows. The reference is the whole model in fp64 over the
final sequence, as in test_gpu_decode.py, whose bound is used: a logit's error reaches 0.235 of the row's standard
deviation, so a token that is among the first k of the GPU's logits is at most twice that, 0.47, below the k-th
largest of the exact ones.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.test_gpu_decode import norm

pytestmark = pytest.mark.gpu


def logits64(d, tokens):
    """test_gpu_decode's model with capped scores."""
    def f(t):
        return t.double().cpu().numpy()
    n = len(tokens)
    x = f(d.embed)[tokens]
    D, hq, h = d.head_dim, d.q_heads, d.heads
    ang = np.arange(n)[:, None, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
    mask = np.tril(np.ones((n, n), dtype=bool))
    for layer in range(d.layers):
        rows = (norm(x) @ f(d.qkv[layer])).reshape(n, hq + 2 * h, D)
        q, k = oc.rotate(rows[:, :hq], ang, False), oc.rotate(rows[:, hq:hq + h], ang, False)
        att = np.empty((n, hq, D))
        for g in range(hq):
            s = q[:, g] @ k[:, g // (hq // h)].T * D ** -0.5
            if d.cap:
                s = d.cap * np.tanh(s / d.cap)
            s = np.where(mask, s, -np.inf)
            w = np.exp(s - s.max(-1, keepdims=True))
            att[:, g] = w @ rows[:, hq + h + g // (hq // h)] / w.sum(-1, keepdims=True)
        x = x + att.reshape(n, -1) @ f(d.out[layer])
    return norm(x) @ f(d.unembed)


@pytest.mark.parametrize("cap", [0.0, 2.0])
def test_emitted_tokens_are_of_the_filtered_target(cap):
    from speculative_decoding_verification_35_gb300 import decode
    B, n, steps = 3, 21, 12
    # fewer pages than the sequences could fill: what a step leaves unused goes back
    d = decode.Decoder(B, n + 1 + steps * (decode.DEPTH + 1) + decode.DEPTH, cap=cap, pages=16)
    g = torch.Generator("cuda").manual_seed(5)
    d.prompt(torch.randint(d.vocab, (B, n), device="cuda", generator=g))
    top_k = [5, 20, 1]
    filters = d.filters(0.9, top_k, [1.0, 0.9, 1.0])
    for _ in range(steps):
        d.sampled_step(filters, 0.9, seed=7, generator=g)
    torch.cuda.synchronize()
    assert int(d.status.item()) == 0 and d.cache.status_bits() == 0 and d.pool.status_bits() == 0
    assert [f.status_bits() for f in filters] == [0, 0, 0]
    lengths = d.lengths.tolist()
    assert d.cached.tolist() == [x - 1 for x in lengths]  # the last emitted token is the next step's first
    assert all(n + 1 + steps <= x for x in lengths)
    assert sum(lengths) > B * (n + 1 + steps)  # some drafts were accepted
    for b in range(B):
        tokens = d.history[b, :lengths[b]].cpu().numpy()
        z = logits64(d, tokens[:-1])[n:]  # (the prompt's own next token is its greedy choice)
        chosen = z[np.arange(len(z)), tokens[n + 1:]]
        least = np.sort(z, -1)[:, -top_k[b]]
        assert (least - chosen <= 0.47 * z.std()).all(), (b, (least - chosen).max())
    # every page has one owner, and the sequences have what their last chunk asked for at most
    held, table = d.pool.held.cpu().numpy(), d.pool.page_table.cpu().numpy()
    head, count = d.pool.state.tolist()
    queue = d.pool.queue.cpu().numpy()
    free = queue[(head + np.arange(count)) % len(queue)]
    assert sorted(np.concatenate([table[b, :held[b]] for b in range(B)] + [free])) == list(range(len(queue)))
    for b in range(B):
        assert -(-(lengths[b] - 1) // 16) <= held[b] <= -(-(lengths[b] + decode.DEPTH) // 16)


def test_ended_sequences_give_their_pages_back():
    from speculative_decoding_verification_35_gb300 import decode
    d = decode.Decoder(2, 64, pages=8)
    d.prompt(torch.randint(d.vocab, (2, 21), device="cuda", generator=torch.Generator("cuda").manual_seed(5)))
    assert d.pool.held.tolist() == [2, 2]
    assert d.pool.reserve(lengths=torch.tensor([0, 21], dtype=torch.int32, device="cuda")) == 0
    assert d.pool.held.tolist() == [0, 2] and d.pool.state.tolist() == [4, 6] and d.pool.status_bits() == 0


def test_command():
    from speculative_decoding_verification_35_gb300 import decode
    assert decode.main(["2", "3", "sample"]) == 0
