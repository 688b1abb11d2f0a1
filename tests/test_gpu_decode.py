"""Generation with token trees over the paged cache: every emitted token is the model's own greedy choice.

The reference is the whole model in fp64 over the final sequence (its roundings of weights and embeddings kept). The
GPU's logits differ from it by the roundings to bfloat16 on the way: per layer the normed input, the projected and
rotated rows, the weights and outputs of the attention and its projection, six or so, and three at the end, each half
a step 2^-8 of a value of its row's size. They add up as independent errors do at worst as their sum: with two layers
fifteen roundings, each passed on with a gain of about one to logits of standard deviation one, 15 x 2^-8 = 0.06 a
standard deviation; a logit's error is taken to reach four of them, so a token may be chosen whose own logit is up to
twice that, 0.47, below the largest.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu


def norm(x):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + np.finfo(np.float32).eps)


def logits64(d, tokens):
    """The model's logits over one sequence, fp64."""
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
            s = np.where(mask, q[:, g] @ k[:, g // (hq // h)].T * D ** -0.5, -np.inf)
            w = np.exp(s - s.max(-1, keepdims=True))
            att[:, g] = w @ rows[:, hq + h + g // (hq // h)] / w.sum(-1, keepdims=True)
        x = x + att.reshape(n, -1) @ f(d.out[layer])
    return norm(x) @ f(d.unembed)


@pytest.mark.parametrize("heads", [2, 8])
def test_trees_generate_the_greedy_sequence(heads):
    from speculative_decoding_verification_35_gb300 import decode
    n, steps = 21, 12
    d = decode.Decoder(3, n + 1 + steps * (decode.DEPTH + 1) + len(decode.PARENTS), heads=heads)
    g = torch.Generator("cuda").manual_seed(5)
    d.prompt(torch.randint(d.vocab, (3, n), device="cuda", generator=g))
    for _ in range(steps):
        d.step()
    torch.cuda.synchronize()
    assert int(d.status.item()) == 0 and d.cache.status_bits() == 0
    lengths = d.lengths.tolist()
    # the last emitted token is the next step's root: not in the cache yet
    assert d.cached.tolist() == [x - 1 for x in lengths]
    assert all(n + 1 + steps <= x for x in lengths) and sum(lengths) > 3 * (n + 1 + steps)  # some drafts were accepted
    for b in range(3):
        tokens = d.history[b, :lengths[b]].cpu().numpy()
        z = logits64(d, tokens[:-1])[n - 1:]
        chosen = z[np.arange(len(z)), tokens[n:]]
        assert (z.max(-1) - chosen <= 0.47 * z.std()).all(), (z.max(-1) - chosen).max()


def test_command():
    from speculative_decoding_verification_35_gb300 import decode
    assert decode.main(["2", "3"]) == 0
