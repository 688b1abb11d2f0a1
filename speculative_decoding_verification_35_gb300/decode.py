"""A small decoder that generates with token trees, or samples: the calls as they are used together.

    python -m speculative_decoding_verification_35_gb300.decode [SEQUENCES] [STEPS] [sample [CAP]]

The target model is a few layers of attention over a paged cache, with random weights (projections are torch
products) and, if wanted, capped scores. A step makes room for its tokens in the cache (spec_cache_reserve), drafts a
token tree per sequence, runs the model once over the trees (in every layer spec_cache_append and spec_cache_attend),
verifies them (spec_verify_tree), moves the accepted paths to the front of their slots (spec_cache_compact) and appends
the emitted tokens to the histories (spec_verify_commit). The drafts come from the model without its layers, a bigram
table: the best WIDTH children of the root, and below each of them the best continuation, DEPTH tokens deep. A sampled
step draws a chain of DEPTH drafts from the bigram's filtered distributions (spec_sample), filters the target's and the
drafts' logits (spec_filter) and verifies them as they are then (spec_verify_fused). No step waits for the host. The prompt
is a chunk like any other, a chain whose tokens are all kept.
"""
from __future__ import annotations

import ctypes
import sys

import torch

from . import speccache as sc
from . import specsample as ss
from . import specverify as sv

WIDTH, DEPTH = 3, 3
# node 0 is the root, nodes 1 .. WIDTH its children, and each further level continues the one before it
PARENTS = [0] * WIDTH + [j - WIDTH for j in range(WIDTH + 1, WIDTH * DEPTH + 1)]


def _ok(rc):
    if rc != sv.SV_OK:
        raise RuntimeError(sv.spec_verify_status_string(rc))


class Filters(tuple):
    """A sampled step's filters of the batch, its draft rows and its target rows; temperature: what their rows are verified
    with, None if any will do."""

    def __new__(cls, filters, temperature):
        self = super().__new__(cls, filters)
        self.temperature = temperature
        return self


class Decoder:
    """Random-weight decoder over a paged cache. dim: of the residual stream; heads: key and value heads; cap: of the
    attention's scores, 0 for none; pages: of the pool, as many as all sequences can fill by default."""

    def __init__(self, sequences, capacity, vocab=512, dim=256, layers=2, q_heads=8, heads=2, head_dim=64, page_size=16,
                 seed=0, device="cuda", cap=0.0, pages=None):
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
        pages = sequences * per if pages is None else pages
        self.cap = cap
        self.pool = sc.PagePool.create(sequences, per, pages, page_size, device)
        shape = (layers, pages, page_size, heads, head_dim)
        self.cache = sc.PagedCache(torch.empty(shape, dtype=torch.bfloat16, device=device),
                                   torch.empty(shape, dtype=torch.bfloat16, device=device), self.pool.page_table)
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
        # a sampled step's chain, its tokens and the logits of its drafts
        self.chain_offs = torch.arange(sequences + 1, **i32) * DEPTH
        self.chain_gammas = torch.full((sequences,), DEPTH, **i32)
        self.chain = sc.Chunk(self.chain_offs, self.cached, sequences * (DEPTH + 1), DEPTH)
        self.steps = 0
        self.ws_bytes = sv.spec_verify_workspace_size(sequences, vocab, n)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=device)

    @staticmethod
    def _norm(x):
        return torch.nn.functional.rms_norm(x, x.shape[-1:]).to(torch.bfloat16)

    def forward(self, chunk, tokens):
        """Logits (bfloat16) of a chunk's rows; its keys and values are appended to the cache, in pages that are taken for
        them (and of those that the last chunk took, the ones that it left unused go back)."""
        _ok(self.pool.reserve(chunk))
        x = self.embed[tokens].float()
        D, hq, h = self.head_dim, self.q_heads, self.heads
        q_rot = torch.empty((len(tokens), hq, D), dtype=torch.bfloat16, device=x.device)
        att = torch.empty_like(q_rot)
        for layer in range(self.layers):
            rows = (self._norm(x) @ self.qkv[layer]).view(-1, hq + 2 * h, D)
            _ok(self.cache.append(chunk, rows[:, :hq], rows[:, hq:hq + h], rows[:, hq + h:], q_rot, self.rope, layer))
            _ok(self.cache.attend(chunk, q_rot, att, layer=layer, cap=self.cap))
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


    def filters(self, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
        """The filters of a sampled step's draft and target rows; each argument a number, or one a sequence. The sequences
        are verified by one call, which has one temperature: theirs are the same, or 0."""
        def each(x, kind):
            return torch.as_tensor(x, dtype=kind, device=self.cached.device).expand(self.B).contiguous()
        given = sorted(set(each(temperature, torch.float32).tolist()) - {0.0})
        if len(given) > 1:
            raise ValueError(f"one verify call has one temperature (or 0 for some sequences), got {given}")
        asked = (each(temperature, torch.float32), each(top_k, torch.int32), each(top_p, torch.float32),
                 each(min_p, torch.float32))
        who = torch.arange(self.B, dtype=torch.int32, device=self.cached.device)
        return Filters((ss.Filter(*asked), ss.Filter(*asked, request=who.repeat_interleave(DEPTH)),
                        ss.Filter(*asked, request=who.repeat_interleave(DEPTH + 1))), given[0] if given else None)

    def sampled_step(self, filters, temperature, seed=0, generator=None):
        """Drafts, verifies and keeps up to DEPTH + 1 new tokens a sequence, drawn from the target's filtered
        distributions. filters: of `filters`, with this temperature."""
        if filters.temperature not in (None, ctypes.c_float(temperature).value):
            raise ValueError(f"the filters' temperature is {filters.temperature}, got {temperature}")
        B, dev = self.B, self.cached.device
        drafts = torch.empty((B, DEPTH), dtype=torch.int32, device=dev)
        logits = torch.empty((B, DEPTH, self.vocab), dtype=torch.bfloat16, device=dev)
        token, drawn = self.next, torch.empty(B, dtype=torch.int32, device=dev)
        for j in range(DEPTH):
            logits[:, j] = self._norm(self.embed[token].float()) @ self.unembed
            _ok(filters[0].sample(logits[:, j], torch.rand(B, generator=generator, device=dev), drawn))
            drafts[:, j] = drawn
            token = drawn
        target = self.forward(self.chain, torch.cat((self.next[:, None], drafts), 1).reshape(-1))
        draft = logits.view(B * DEPTH, self.vocab)
        _ok(filters[1].mask(draft, draft))
        _ok(filters[2].mask(target, target))
        self.steps += 1
        _ok(sv.spec_verify_fused(target.data_ptr(), draft.data_ptr(), sv.SV_BF16, drafts.data_ptr(), self.chain_offs.data_ptr(),
                                 self.chain_gammas.data_ptr(), B, self.vocab, DEPTH, temperature, seed, self.steps,
                                 self.tokens_out.data_ptr(), self.accepted.data_ptr(), self.status.data_ptr(), self.ws.data_ptr(),
                                 self.ws_bytes, self.history.data_ptr(), self.capacity, self.lengths.data_ptr(), self.next.data_ptr(),
                                 torch.cuda.current_stream().cuda_stream))
        _ok(self.cache.compact(self.chain, self.accepted, None, self.cached))


def main(argv=None) -> int:
    argv = sys.argv[1:] if argv is None else argv
    B = int(argv[0]) if argv else 4
    steps = int(argv[1]) if len(argv) > 1 else 32
    sampled = len(argv) > 2 and argv[2] == "sample"
    cap = float(argv[3]) if len(argv) > 3 else 0.0
    n = 20
    d = Decoder(B, n + 1 + steps * (DEPTH + 1) + len(PARENTS), cap=cap)
    d.prompt(torch.randint(d.vocab, (B, n), device="cuda", generator=torch.Generator("cuda").manual_seed(1)))
    filters = d.filters(0.8, 50, 0.95, 0.01)
    for _ in range(steps):
        if sampled:
            d.sampled_step(filters, 0.8, generator=torch.Generator("cuda").manual_seed(d.steps))
        else:
            d.step()
    torch.cuda.synchronize()
    found = [int(d.status.item()), d.cache.status_bits(), d.pool.status_bits()] + [f.status_bits() for f in filters]
    if any(found):
        print("device status", *found, file=sys.stderr)
        return 1
    got = d.lengths - n - 1
    print(f"{B} sequences, {steps} steps: {got.tolist()} tokens, {got.float().mean().item() / steps:.2f} a step")
    print("sequence 0:", d.history[0, n:n + 1 + int(got[0])].tolist())
    return 0


if __name__ == "__main__":
    sys.exit(main())
