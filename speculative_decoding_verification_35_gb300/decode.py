"""A small decoder that generates with token trees: the cache calls and the verify step as they are used together.

    python -m speculative_decoding_verification_35_gb300.decode [SEQUENCES] [STEPS]

The target model is a few layers of attention over a paged cache, with random weights (projections are torch
products). A step drafts a token tree per sequence, runs the model once over the trees (in every layer
spec_cache_append and spec_cache_attend), verifies them (spec_verify_tree), moves the accepted paths to the front of
their slots (spec_cache_compact) and appends the emitted tokens to the histories (spec_verify_commit). The drafts come
from the model without its layers, a bigram table: the best WIDTH children of the root, and below each of them the
best continuation, DEPTH tokens deep. No step waits for the host. The prompt is a chunk like any other, a chain whose
tokens are all kept.
"""
from __future__ import annotations

import sys

import torch

from . import speccache as sc
from . import specverify as sv

WIDTH, DEPTH = 3, 3
# node 0 is the root, nodes 1 .. WIDTH its children, and each further level continues the one before it
PARENTS = [0] * WIDTH + [j - WIDTH for j in range(WIDTH + 1, WIDTH * DEPTH + 1)]


def _ok(rc):
    if rc != sv.SV_OK:
        raise RuntimeError(sv.spec_verify_status_string(rc))


class Decoder:
    """Random-weight decoder over a paged cache. dim: of the residual stream; heads: key and value heads."""

    def __init__(self, sequences, capacity, vocab=512, dim=256, layers=2, q_heads=8, heads=2, head_dim=64, page_size=16,
                 seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, m):
            return (torch.randn((n, m), generator=g, device=device) * n ** -0.5).to(torch.bfloat16)
        self.B, self.capacity, self.vocab, self.layers = sequences, capacity, vocab, layers
        self.q_heads, self.heads, self.head_dim = q_heads, heads, head_dim
        self.embed = torch.randn((vocab, dim), generator=g, device=device).to(torch.bfloat16)
        self.qkv = [weight(dim, (q_heads + 2 * heads) * head_dim) for _ in range(layers)]
        self.out = [weight(q_heads * head_dim, dim) for _ in range(layers)]
        self.unembed = weight(dim, vocab)
        angles = torch.arange(capacity, device=device)[:, None] * 10000.0 ** (
            -torch.arange(0, head_dim, 2, device=device) / head_dim)
        self.rope = sc.Rope(torch.cat((angles.cos(), angles.sin()), 1).float())
        per = -(-capacity // page_size)
        pages = torch.randperm(sequences * per, generator=g, device=device).to(torch.int32)
        shape = (layers, sequences * per, page_size, heads, head_dim)
        self.cache = sc.PagedCache(torch.empty(shape, dtype=torch.bfloat16, device=device),
                                   torch.empty(shape, dtype=torch.bfloat16, device=device), pages.view(sequences, per))
        i32 = dict(dtype=torch.int32, device=device)
        self.cached = torch.zeros(sequences, **i32)
        self.history = torch.zeros((sequences, capacity), **i32)
        self.lengths = torch.zeros(sequences, **i32)
        self.next = torch.zeros(sequences, **i32)
        self.accepted = torch.zeros(sequences, **i32)
        self.status = torch.zeros(1, **i32)
        n = len(PARENTS)
        self.offs = torch.arange(sequences + 1, **i32) * n
        self.gammas = torch.full((sequences,), n, **i32)
        self.parents = torch.tensor(PARENTS * sequences, **i32)
        self.path = torch.empty(sequences * n, **i32)
        self.tokens_out = torch.empty(sequences * (n + 1), **i32)
        self.tree = sc.Chunk(self.offs, self.cached, sequences * (n + 1), n, self.parents)
        self.ws_bytes = sv.spec_verify_workspace_size(sequences, vocab, n)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=device)

    @staticmethod
    def _norm(x):
        return torch.nn.functional.rms_norm(x, x.shape[-1:]).to(torch.bfloat16)

    def forward(self, chunk, tokens):
        """Logits (bfloat16) of a chunk's rows; its keys and values are appended to the cache."""
        x = self.embed[tokens].float()
        D, hq, h = self.head_dim, self.q_heads, self.heads
        q_rot = torch.empty((len(tokens), hq, D), dtype=torch.bfloat16, device=x.device)
        att = torch.empty_like(q_rot)
        for layer in range(self.layers):
            rows = (self._norm(x) @ self.qkv[layer]).view(-1, hq + 2 * h, D)
            _ok(self.cache.append(chunk, rows[:, :hq], rows[:, hq:hq + h], rows[:, hq + h:], q_rot, self.rope, layer))
            _ok(self.cache.attend(chunk, q_rot, att, layer=layer))
            x = x + (att.view(len(tokens), -1) @ self.out[layer]).float()
        return self._norm(x) @ self.unembed

    def prompt(self, tokens):
        """Starts every sequence with a prompt, int [sequences, n]."""
        B, n = tokens.shape
        i32 = dict(dtype=torch.int32, device=tokens.device)
        offs, gammas = torch.arange(B + 1, **i32) * (n - 1), torch.full((B,), n - 1, **i32)
        self.cached.zero_()
        chunk = sc.Chunk(offs, self.cached, B * n, n - 1)
        logits = self.forward(chunk, tokens.reshape(-1))
        self.cached += n  # a chain, all of it kept
        self.next.copy_(logits.view(B, n, -1)[:, -1].argmax(-1))
        self.history[:, :n] = tokens
        self.history[:, n] = self.next
        self.lengths.fill_(n + 1)

    def draft(self):
        """The trees' tokens, root first, [sequences, nodes]."""
        def after(t):
            return self._norm(self.embed[t].float()) @ self.unembed
        level = after(self.next).topk(WIDTH, -1).indices
        nodes = [self.next[:, None], level]
        for _ in range(DEPTH - 1):
            level = after(level).argmax(-1)
            nodes.append(level)
        return torch.cat(nodes, 1)

    def step(self):
        """Drafts, verifies and keeps: up to DEPTH + 1 new tokens a sequence."""
        tree = self.draft()
        logits = self.forward(self.tree, tree.reshape(-1))
        drafts = tree[:, 1:].to(torch.int32).contiguous()
        stream = torch.cuda.current_stream().cuda_stream
        n, status = len(PARENTS), self.status.data_ptr()
        _ok(sv.spec_verify_tree(logits.data_ptr(), sv.SV_BF16, drafts.data_ptr(), self.parents.data_ptr(), self.offs.data_ptr(),
                                self.gammas.data_ptr(), self.B, self.vocab, n, 0.0, 0, 0, self.tokens_out.data_ptr(),
                                self.accepted.data_ptr(), self.path.data_ptr(), status, self.ws.data_ptr(), self.ws_bytes,
                                stream))
        _ok(self.cache.compact(self.tree, self.accepted, self.path, self.cached))
        _ok(sv.spec_verify_commit(self.tokens_out.data_ptr(), self.accepted.data_ptr(), self.offs.data_ptr(), self.B,
                                  self.history.data_ptr(), self.capacity, self.lengths.data_ptr(), self.next.data_ptr(),
                                  status, stream))


def main(argv=None) -> int:
    argv = sys.argv[1:] if argv is None else argv
    B = int(argv[0]) if argv else 4
    steps = int(argv[1]) if len(argv) > 1 else 32
    n = 20
    d = Decoder(B, n + 1 + steps * (DEPTH + 1) + len(PARENTS))
    d.prompt(torch.randint(d.vocab, (B, n), device="cuda", generator=torch.Generator("cuda").manual_seed(1)))
    for _ in range(steps):
        d.step()
    torch.cuda.synchronize()
    if int(d.status.item()) or d.cache.status_bits():
        print("device status", int(d.status.item()), d.cache.status_bits(), file=sys.stderr)
        return 1
    got = d.lengths - n - 1
    print(f"{B} sequences, {steps} steps: {got.tolist()} tokens, {got.float().mean().item() / steps:.2f} a step")
    print("sequence 0:", d.history[0, n:n + 1 + int(got[0])].tolist())
    return 0


if __name__ == "__main__":
    sys.exit(main())
