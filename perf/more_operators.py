"""Cases of the operators around a verify step: sampling, filtered logits, pages from lengths, scored attention.

A decoding step with a draft model samples its drafts from filtered distributions (temperature, top-k, top-p, min-p),
filters the target's and the draft's logits in the same way before they are verified, makes room in the paged cache
for the chunk's tokens, and attends over it with the scores that the model wants: capped by a tanh, biased by
distance, or with a prefix that every token sees.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "fp16": 2, "e4m3": 1}


# ----------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------
def _rows(name, op, rows, V, kind="bf16", filters="kp", sigma=2.5, zipf=1.1, requests=0, pad=0):
    """Logit rows. filters: letters of k, p, m and t that the requests use (t: temperatures other than 1); "mixed":
    every request its own. requests: how many share the rows, 0 for one a row. pad: columns past V in a row."""
    return dict(name=name, op=op, rows=rows, V=V, kind=kind, filters=filters, sigma=sigma, zipf=zipf,
                requests=requests, pad=pad)


def _pages(name, B, chunk, chunk_min, ctx, ctx_min, page, mode="chunk", lens=1):
    """chunk, ctx: largest tokens of a chunk and largest cached length. mode "chunk": room for the chunk and its slot
    map; "lengths": room for given lengths, some of them zero (sequences that have ended)."""
    return dict(name=name, op="reserve", B=B, chunk=chunk, chunk_min=chunk_min, ctx=ctx, ctx_min=ctx_min, page=page,
                mode=mode, lens=lens)


def _attend(name, B, chunk, chunk_min, ctx, ctx_min, hq, hkv, d, page, kind="bf16", cache="bf16", order="token",
            tree=False, window=0, cap=0.0, slopes=False, prefix=False, lens=1):
    """order: "token" keeps a page as [page, head, dim] rows, "head" as [head, page, dim]."""
    return dict(name=name, op="attend", B=B, chunk=chunk, chunk_min=chunk_min, ctx=ctx, ctx_min=ctx_min, hq=hq, hkv=hkv,
                d=d, page=page, kind=kind, cache=cache, order=order, tree=tree, window=window, cap=cap, slopes=slopes,
                prefix=prefix, lens=lens)


def listed():
    return [
        # one stream's next draft token: the call's latency
        _rows("sample one row", "sample", 1, 32000, filters="kpt", sigma=3.0),
        # a draft model's tokens for the benchmark's batch, nucleus alone
        _rows("sample 64 rows nucleus", "sample", 64, 128256, filters="p"),
        # a serving batch whose requests all ask for something else, an odd vocabulary in float
        _rows("sample 128 rows mixed f32", "sample", 128, 129281, kind="f32", filters="mixed", sigma=2.0),
        # a small verify batch: 4 drafts and one sequence, float
        _rows("filter 9 rows f32", "filter", 9, 1024, kind="f32", filters="kp", sigma=2.0, zipf=0.0, requests=1),
        # the rows of 8 sequences with 4 drafts, target and draft
        _rows("filter 72 rows", "filter", 72, 32000, filters="kpt", sigma=3.0, requests=8),
        # the rows of the benchmark's verify batch (64 sequences, 5 drafts), a filter for each sequence
        _rows("filter 704 rows mixed", "filter", 704, 128256, filters="mixed", requests=64),
        # a verify batch crosses into new pages
        _pages("reserve verify 64x6", 64, 6, 6, 8000, 500, 16),
        # prompts come in, with their slots
        _pages("reserve prompts 32", 32, 8192, 700, 60000, 1, 16),
        # plain decoding of one stream with capped scores
        _attend("attend capped one token", 1, 1, 1, 900, 900, 32, 8, 128, 16, cap=50.0),
        # the benchmark's verify batch in a capped local layer
        _attend("attend capped verify 64x6", 64, 6, 6, 8000, 500, 32, 8, 128, 16, cap=50.0, window=4096),
        # token trees with a bias by distance, heads of their own
        _attend("attend distance trees 16x32", 16, 32, 32, 4001, 300, 16, 16, 64, 32, kind="fp16", cache="fp16",
                order="head", tree=True, slopes=True),
        # prompts with a prefix that all tokens see, capped: bound by products and exponentials
        _attend("attend prefix prompts 3x2048", 3, 2048, 700, 8192, 1, 32, 8, 128, 64, cap=30.0, prefix=True),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "filter", "filter", "reserve", "attend", "attend", "attend"])
    if op in ("sample", "filter"):
        V = _between(rng, 1000, 152064)
        rows = _between(rng, 1, min(256, 12_000_000 // V))
        c = _rows("", op, rows, V, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["k", "p", "kp", "kpt", "mt", "mixed", "mixed"]),
                  rng.choice([1.5, 2.0, 2.5, 3.0]), rng.choice([0.0, 1.05, 1.1]),
                  rng.choice([0, _between(rng, 1, rows)]), rng.choice([0, 0, rng.randrange(1, 64)]))
    elif op == "reserve":
        chunk = _between(rng, 1, 4096)
        ctx = _between(rng, 1, 30000)
        c = _pages("", _between(rng, 1, max(1, min(512, 600_000 // (chunk + ctx)))), chunk, _between(rng, 1, chunk), ctx,
                   _between(rng, 1, ctx), rng.choice([8, 16, 32, 48, 64, 128]), rng.choice(["chunk", "chunk", "lengths"]),
                   rng.randrange(1 << 20))
    else:
        hkv = rng.choice([1, 2, 3, 4, 8])
        kind = rng.choice(["bf16", "bf16", "fp16"])
        shape = rng.choice(["tokens", "drafts", "drafts", "trees", "prompts"])
        if shape == "prompts":
            chunk, B, ctx = _between(rng, 33, 2048), _between(rng, 1, 3), _between(rng, 1, 8192)
        else:
            chunk, B = 1 if shape == "tokens" else rng.randrange(2, 33), _between(rng, 1, 64)
            ctx = min(65536, _between(rng, 1, 300000 // B))
        score = rng.choice(["cap", "cap", "distance", "both", "prefix", "prefix and cap"])
        c = _attend("", B, chunk, _between(rng, 1, chunk), ctx, _between(rng, 1, ctx), hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]),
                    hkv, rng.choice([64, 128, 128, 80, 96]), rng.choice([8, 16, 32, 48, 64, 128]), kind,
                    rng.choice([kind, kind, "e4m3"]) if kind == "bf16" else kind, rng.choice(["token", "head"]),
                    shape == "trees" and "prefix" not in score, rng.choice([0, 0, 0, _between(rng, 16, 4096)]),
                    rng.choice([20.0, 30.0, 50.0]) if "cap" in score or score == "both" else 0.0,
                    score in ("distance", "both"), "prefix" in score, rng.randrange(1 << 20))
    del c["name"]
    return c


# ----------------------------------------------------------------------------------------------------------
# what the lengths of a case are
# ----------------------------------------------------------------------------------------------------------
def _lengths(case):
    """(chunk lengths, cached lengths, what the op's own draws need)."""
    rng = random.Random(case["lens"])
    B = case["B"]
    chunk = [_between(rng, case["chunk_min"], case["chunk"]) for _ in range(B)]
    cached = [_between(rng, case["ctx_min"], case["ctx"]) for _ in range(B)]
    chunk[0], cached[-1] = case["chunk"], case["ctx"]  # the largest are there
    return chunk, cached, rng


def _held(case):
    """(lengths to hold, pages held) of each sequence of a reserve call."""
    chunk, cached, rng = _lengths(case)
    page = case["page"]
    want = [p + n for n, p in zip(chunk, cached)]
    held = []
    for b, past in enumerate(cached):
        if case["mode"] == "lengths" and rng.random() < 0.15:
            want[b] = 0  # it has ended
        # what the last step's chunk had asked for: some sequences have a page or two more than they need now
        held.append(-(-(past + rng.choice([0, 0, 0, page, 2 * page])) // page))
    return want, held


def _parents(case, chunk, rng):
    return [[max(0, rng.randrange(j) - rng.randrange(3)) for j in range(1, n)] for n in chunk] if case["tree"] else None


def _depths(par):
    dep = [0]
    for p in par:
        dep.append(dep[p] + 1)
    return dep


def _prefixes(case, chunk, cached, rng):
    """Slots that all tokens of a sequence see: into the chunk for some, within what is cached for others."""
    return [rng.randrange(0, p + n + n // 2 + 1) for n, p in zip(chunk, cached)] if case["prefix"] else None


def work(case):
    if case["op"] in ("sample", "filter"):
        n = case["rows"] * case["V"]
        # each logit in (filter: and out), a row's parameters and results; an exponential and its sum a logit
        return {"bytes": n * SIZE[case["kind"]] * (2 if case["op"] == "filter" else 1) + 32 * case["rows"], "flops": 4 * n}
    chunk, cached, rng = _lengths(case)
    if case["op"] == "reserve":
        want, held = _held(case)
        moved = sum(abs(-(-n // case["page"]) - h) for n, h in zip(want, held))
        slots = sum(chunk) if case["mode"] == "chunk" else 0
        touched = sum(-(-n // case["page"]) + 1 for n in chunk) if slots else 0
        return {"bytes": 8 * moved + 8 * slots + 4 * touched + 16 * case["B"], "flops": 0}
    parents = _parents(case, chunk, rng)
    prefixes = _prefixes(case, chunk, cached, rng)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    a, c = SIZE[case["kind"]], SIZE[case["cache"]]
    seen = tokens = 0
    w = case["window"] or 1 << 30
    for b, (n, past) in enumerate(zip(chunk, cached)):
        for t in _depths(parents[b]) if parents else range(n):
            first = max(0, past + t - w + 1)
            last = past + t + 1
            if prefixes:
                last = max(last, min(prefixes[b], past + n))
            seen += last - first
        tokens += min(past, w - 1) + n
    return {"bytes": 2 * tokens * hkv * d * c + sum(chunk) * hq * (2 * d * a + 4) + 4 * (tokens // case["page"]),
            "flops": seen * hq * (4 * d + 4)}


# ----------------------------------------------------------------------------------------------------------
# what a program has before the call
# ----------------------------------------------------------------------------------------------------------
def _row_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, V, kind = case["rows"], case["V"], TYPES[case["kind"]]
    # a model's logits: noise and a prior that falls with the token's rank
    prior = -case["zipf"] * torch.arange(1, V + 1, device=DEV).log()
    full = torch.empty((rows, V + case["pad"]), dtype=kind, device=DEV)
    for r in range(0, rows, 64):
        x = torch.randn((min(64, rows - r), V), generator=g, device=DEV) * case["sigma"] + prior
        full[r:r + 64, :V] = x.to(kind)
    full[:, V:] = 30.0  # what lies past the vocabulary is no logit
    n = case["requests"] or rows
    f = case["filters"]
    use = {c: torch.ones(n, dtype=torch.bool, device=DEV) if c in f else torch.zeros(n, dtype=torch.bool, device=DEV) for c in "kpmt"}
    if f == "mixed":
        use = {c: torch.rand(n, generator=g, device=DEV) < 0.6 for c in "kpmt"}
    some = torch.rand((4, n), generator=g, device=DEV)
    s = dict(case=case, logits=full[:, :V], uniforms=torch.rand(rows, generator=g, device=DEV))
    s["top_k"] = torch.where(use["k"], (20 + 180 * some[0]).int(), 0)
    s["top_p"] = torch.where(use["p"], 0.8 + 0.19 * some[1], 1.0)
    s["min_p"] = torch.where(use["m"], 0.02 + 0.1 * some[2], 0.0)
    s["temperature"] = torch.where(use["t"], 0.6 + 0.7 * some[3], 1.0)
    if f == "mixed" and n > 3:
        s["temperature"][n // 2] = 0.0  # one of them greedy
    s["request"] = (torch.arange(rows, device=DEV) * n // rows).int() if case["requests"] else None
    return s


def _page_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    chunk, cached, _ = _lengths(case)
    want, held = _held(case)
    B, page = case["B"], case["page"]
    need = [-(-n // page) for n in want]
    width = max(need + held) + 1
    pages = sum(max(a, b) for a, b in zip(need, held)) + 7
    ints = dict(dtype=torch.int32, device=DEV)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, **ints)
    at = torch.arange(width, device=DEV)
    h = torch.tensor(held, device=DEV)
    mine = at < h[:, None]
    table[mine] = order[:sum(held)]
    free = pages - sum(held)
    head = int(torch.randint(pages, (1,), generator=g, device=DEV))
    queue = torch.full((pages,), -1, **ints)
    queue[(head + torch.arange(free, device=DEV)) % pages] = order[sum(held):]
    s = dict(case=case, table=table, queue=queue, state=torch.tensor([head, free], **ints), held=torch.tensor(held, **ints), pages=pages)
    offs = [0]
    for n in chunk:
        offs.append(offs[-1] + n - 1)
    s["offs"], s["cached"], s["rows"] = torch.tensor(offs, **ints), torch.tensor(cached, **ints), sum(chunk)
    s["lengths"] = torch.tensor(want, **ints) if case["mode"] == "lengths" else None
    return s


def _attend_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    chunk, cached, rng = _lengths(case)
    parents = _parents(case, chunk, rng)
    prefixes = _prefixes(case, chunk, cached, rng)
    B, hq, hkv, d, page = (case[k] for k in ("B", "hq", "hkv", "d", "page"))
    kind, held = TYPES[case["kind"]], TYPES[case["cache"]]
    need = [-(-(n + past) // page) for n, past in zip(chunk, cached)]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)  # a sequence's pages lie anywhere
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n

    def cache():
        y = torch.randn((pages, page, hkv, d) if case["order"] == "token" else (pages, hkv, page, d), generator=g, device=DEV,
                        dtype=torch.float16)
        x = ((y * 60.0) if case["cache"] == "e4m3" else y).to(held)[None]
        return x if case["order"] == "token" else x.transpose(2, 3)

    s = dict(case=case, k_cache=cache(), v_cache=cache(), table=table, k_scale=None, v_scale=None)
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.012 + 0.008 * torch.rand((1, hkv), generator=g, device=DEV)
        s["v_scale"] = 0.012 + 0.008 * torch.rand((1, hkv), generator=g, device=DEV)
    ints = dict(dtype=torch.int32, device=DEV)
    offs = [0]
    for n in chunk:
        offs.append(offs[-1] + n - 1)
    s["offs"], s["cached"] = torch.tensor(offs, **ints), torch.tensor(cached, **ints)
    s["parents"] = torch.tensor(sum(parents, []) or [0], **ints) if parents else None
    s["prefix"] = torch.tensor(prefixes, **ints) if prefixes else None
    # the slopes of models that use them: a geometric series over the heads
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device=DEV) / hq) if case["slopes"] else None
    s["rows"], s["most"] = sum(chunk), case["chunk"]
    s["host"] = (chunk, cached, parents, prefixes)
    if parents:  # each tree's depths, and which nodes lie on the way to a node
        s["trees"] = []
        for par in parents:
            line = torch.eye(len(par) + 1, dtype=torch.bool)
            for j, p in enumerate(par, 1):
                line[j] |= line[p]
            s["trees"].append((torch.tensor(_depths(par), device=DEV), line.to(DEV)))
    s["q"] = (torch.randn((s["rows"], hq, d), generator=g, device=DEV) * 4.0).to(kind)
    s["scale"] = 1.0 / math.sqrt(d)
    return s


def prepare(case, seed):
    if case["op"] in ("sample", "filter"):
        s = _row_inputs(case, seed)
    else:
        s = _page_inputs(case, seed) if case["op"] == "reserve" else _attend_inputs(case, seed)
    if own:  # the program's handles and the outputs' buffers
        ints = dict(dtype=torch.int32, device=DEV)
        if case["op"] in ("sample", "filter"):
            from speculative_decoding_verification_35_gb300 import specsample as ss
            s["filter"] = ss.Filter(s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["request"])
            s["kept"] = torch.empty(case["rows"], **ints)
            if case["op"] == "sample":
                s["tokens"] = torch.empty(case["rows"], **ints)
                s["logprobs"] = torch.empty(case["rows"], device=DEV)
            else:
                s["out"] = torch.empty((case["rows"], case["V"]), dtype=TYPES[case["kind"]], device=DEV)
        else:
            from speculative_decoding_verification_35_gb300 import speccache as sc
            if case["op"] == "reserve":
                s["pool"] = sc.PagePool(s["table"], s["queue"], s["held"], s["state"], case["page"])
                s["out_held"], s["out_state"] = torch.empty_like(s["held"]), torch.empty_like(s["state"])
                if s["lengths"] is None:
                    s["chunk"] = sc.Chunk(s["offs"], s["cached"], s["rows"], case["chunk"] - 1)
                    s["slots"] = torch.empty(s["rows"], dtype=torch.int64, device=DEV)
            else:
                s["cache"] = sc.PagedCache(s["k_cache"], s["v_cache"], s["table"], s["k_scale"], s["v_scale"])
                s["chunk"] = sc.Chunk(s["offs"], s["cached"], s["rows"], s["most"] - 1, s["parents"])
                s["out"] = torch.empty((s["rows"], case["hq"], case["d"]), dtype=TYPES[case["kind"]], device=DEV)
                s["lse"] = torch.empty((s["rows"], case["hq"]), device=DEV)
    return s


# ----------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------
def _done(rc):
    if rc != 0:
        raise RuntimeError("status %d" % rc)


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"sample": _sample, "filter": _filter, "reserve": _reserve, "attend": _attention}[op](s)
    if op == "sample":
        _done(s["filter"].sample(s["logits"], s["uniforms"], s["tokens"], s["logprobs"], s["kept"]))
        return s["tokens"], s["logprobs"], s["kept"]
    if op == "filter":
        _done(s["filter"].mask(s["logits"], s["out"], s["kept"]))
        return s["out"], s["kept"]
    if op == "reserve":
        if s["lengths"] is not None:
            _done(s["pool"].reserve(lengths=s["lengths"], out_held=s["out_held"], out_state=s["out_state"]))
            return s["table"], s["queue"], s["out_held"], s["out_state"]
        _done(s["pool"].reserve(chunk=s["chunk"], slot_map=s["slots"], out_held=s["out_held"], out_state=s["out_state"]))
        return s["table"], s["queue"], s["out_held"], s["out_state"], s["slots"]
    _done(s["cache"].attend(s["chunk"], s["q"], s["out"], s["lse"], scale=s["scale"], window=case["window"], cap=case["cap"],
                            slopes=s["slopes"], prefix=s["prefix"]))
    return s["out"], s["lse"]


# Rows, in 64 bits: which tokens are kept, and which one is drawn, is decided next to borders.
def _kept(s, a, b):
    """(weights, kept) of the rows a .. b - 1, [rows, V], in the vocabulary's order."""
    l = s["logits"][a:b].double()
    req = torch.arange(a, b, device=DEV) if s["request"] is None else s["request"][a:b].long()
    T, k, p, mp = (s[n][req][:, None] for n in ("temperature", "top_k", "top_p", "min_p"))
    p, mp = p.double(), mp.double()
    w = ((l - l.amax(1, keepdim=True)) / torch.where(T > 0, T, torch.ones_like(T)).double()).exp()
    order = l.sort(dim=1, descending=True, stable=True).indices  # ties: the lowest index first
    rank = torch.arange(l.shape[1], device=DEV)
    first = rank[None] == 0
    ws = w.gather(1, order)
    ok = (rank < torch.where(k > 0, k, l.shape[1])) & (ws > 0)
    ws = ws * ok
    sums = ws.cumsum(1)
    before = torch.cat((torch.zeros_like(sums[:, :1]), sums[:, :-1]), 1)
    ok &= (p >= 1) | (before < p * sums[:, -1:]) | first
    ok &= (ws >= mp) | first
    ok &= (T > 0) | first
    keep = torch.zeros_like(ok).scatter(1, order, ok)
    return w, keep


def _filter(s):
    out, kept = [], []
    for a in range(0, s["case"]["rows"], 64):
        x = s["logits"][a:a + 64]
        _, keep = _kept(s, a, a + len(x))
        out.append(torch.where(keep, x, torch.full_like(x, -math.inf)))
        kept.append(keep.sum(1).int())
    return torch.cat(out), torch.cat(kept)


def _sample(s):
    tokens, logprobs, kept = [], [], []
    for a in range(0, s["case"]["rows"], 64):
        u = s["uniforms"][a:a + 64].double()[:, None]
        w, keep = _kept(s, a, a + len(u))
        w = w * keep
        sums = w.cumsum(1)
        total = sums[:, -1:]
        t = (sums <= u * total).sum(1, keepdim=True)
        last = w.shape[1] - 1 - (w > 0).flip(1).int().argmax(1, keepdim=True)
        t = torch.minimum(t, last)
        n = keep.sum(1)
        tokens.append(t[:, 0].int())
        logprobs.append((w.gather(1, t) / total).log()[:, 0].float())
        kept.append(n.int())
    return torch.cat(tokens), torch.cat(logprobs), torch.cat(kept)


def _reserve(s):
    c = s["case"]
    page, B, pages = c["page"], c["B"], s["pages"]
    n = s["offs"][1:] - s["offs"][:-1] + 1
    want = s["cached"] + n if s["lengths"] is None else s["lengths"]
    need = (want + page - 1) // page
    give, take = (s["held"] - need).clamp(min=0), (need - s["held"]).clamp(min=0)
    head, count = s["state"][0], s["state"][1]
    width = s["table"].shape[1]
    at = torch.arange(width, device=DEV)
    # what is given back, to the queue's end, in the order of the sequences
    back = (at >= need[:, None]) & (at < s["held"][:, None])
    j = back.flatten().cumsum(0).view_as(back) - 1
    s["queue"][((head + count + j) % pages)[back]] = s["table"][back]
    count = count + give.sum()
    # from its front, in that order, as long as there are enough
    upto = take.cumsum(0)
    served = upto <= count
    taken = torch.where(served, upto, 0).amax()
    new = (at >= s["held"][:, None]) & (at < need[:, None]) & served[:, None]
    i = (upto - take)[:, None] + at - s["held"][:, None]
    s["table"][new] = s["queue"][((head + i) % pages)[new]]
    out_held = torch.where(served, need, s["held"]).int()
    out_state = torch.stack(((head + taken) % pages, count - taken)).int()
    if s["lengths"] is not None:
        return s["table"], s["queue"], out_held, out_state
    starts = s["offs"][:-1] + torch.arange(B, device=DEV)
    row = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(starts, row, right=True) - 1
    slot = s["cached"][b] + row - starts[b]
    id = s["table"][b, (slot // page).long()].long()
    return s["table"], s["queue"], out_held, out_state, torch.where(served[b], id * page + slot % page, -1)


def _seen(s, b):
    """Sequence b: (slots, which of them each token sees, distances), [T, slots]."""
    chunk, cached, parents, prefixes = s["host"]
    n, past = chunk[b], cached[b]
    slot = torch.arange(past + n, device=DEV)
    if parents:
        dep, line = s["trees"][b]
        pos = torch.cat((slot[:past], past + dep))
        seen = torch.cat((torch.ones((n, past), dtype=torch.bool, device=DEV), line), 1)
    else:
        pos = slot
        seen = slot <= slot[past:, None]
    if prefixes:
        seen = seen | (slot < prefixes[b])
    apart = pos[past:, None] - pos[None]
    if s["case"]["window"]:
        seen = seen & (apart < s["case"]["window"])
    return slot, seen, apart.abs()


def _attention(s):
    c = s["case"]
    chunk = s["host"][0]
    G, page = c["hq"] // c["hkv"], c["page"]
    out = torch.empty((s["rows"], c["hq"], c["d"]), dtype=TYPES[c["kind"]], device=DEV)
    lse = torch.empty((s["rows"], c["hq"]), device=DEV)
    row = 0
    for b, n in enumerate(chunk):
        slot, seen, apart = _seen(s, b)
        at = s["table"][b, slot // page].long() * page + slot % page
        k = s["k_cache"][0][at // page, at % page].float()
        v = s["v_cache"][0][at // page, at % page].float()
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"][0][:, None], v * s["v_scale"][0][:, None]
        q = s["q"][row:row + n].float().view(n, c["hkv"], G, c["d"])
        z = torch.einsum("thgd,shd->hgts", q, k) * s["scale"]
        if c["cap"]:
            z = c["cap"] * (z / c["cap"]).tanh()
        if s["slopes"] is not None:
            z = z - s["slopes"].view(c["hkv"], G, 1, 1) * apart
        z = z.masked_fill(~seen, -math.inf)
        top = z.amax(3, keepdim=True)
        w = (z - top).exp()
        total = w.sum(3, keepdim=True)
        out[row:row + n] = (torch.einsum("hgts,shd->hgtd", w, v) / total).permute(2, 0, 1, 3).flatten(1, 2).to(out.dtype)
        lse[row:row + n] = (top + total.log())[..., 0].permute(2, 0, 1).flatten(1)
        row += n
    return out, lse


# ----------------------------------------------------------------------------------------------------------
# from the definitions, in 64 bits
# ----------------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("sample", "filter"):
        return _exact_rows(case, seed) if case["rows"] * case["V"] <= 4e7 else None
    if case["op"] == "attend":
        return _exact_attend(case, seed)
    return None  # whole numbers alone


def _exact_rows(case, seed):
    """Row by row on the host, each by the ranking itself."""
    s = _row_inputs(case, seed)
    host = {n: s[n].cpu().numpy() for n in ("top_k", "top_p", "min_p", "temperature", "uniforms")}
    which = range(case["rows"]) if s["request"] is None else s["request"].tolist()
    masks, tokens, logprobs, counts = [], [], [], []
    for r, q in enumerate(which):
        l = s["logits"][r].double().cpu().numpy()
        T = float(host["temperature"][q])
        rank = np.lexsort((np.arange(len(l)), -l))
        if T == 0:
            n, w = 1, np.ones(1)
        else:
            w = np.exp((l[rank] - l[rank[0]]) / T)
            n = int(np.count_nonzero(w))
            if 0 < host["top_k"][q] < n:
                n = int(host["top_k"][q])
            if host["top_p"][q] < 1:
                c = np.cumsum(w[:n])
                n = min(n, int(np.searchsorted(c, float(host["top_p"][q]) * c[-1], side="left")) + 1)
            n = max(1, min(n, int(np.searchsorted(-w, -float(host["min_p"][q]), side="right"))))
        counts.append(n)
        if case["op"] == "filter":
            x = np.full(len(l), -np.inf)
            x[rank[:n]] = l[rank[:n]]
            masks.append(torch.from_numpy(x))
            continue
        by = np.argsort(rank[:n])
        c = np.cumsum(w[:n][by])
        i = min(int(np.searchsorted(c, float(host["uniforms"][r]) * c[-1], side="right")), n - 1)
        tokens.append(int(rank[:n][by][i]))
        logprobs.append(math.log(w[:n][by][i] / c[-1]))
    counts = torch.tensor(counts, dtype=torch.int32)
    if case["op"] == "filter":
        return torch.stack(masks), counts
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(logprobs, dtype=torch.float64), counts


def _exact_attend(case, seed):
    """A head at a time, a few hundred tokens at a time."""
    s = _attend_inputs(case, seed)
    if work(case)["flops"] > 1.5e12:
        return None
    chunk, cached, parents, prefixes = s["host"]
    G, page, hq = case["hq"] // case["hkv"], case["page"], case["hq"]
    out = torch.zeros((s["rows"], hq, case["d"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["rows"], hq), dtype=torch.float64, device=DEV)
    row = 0
    for b, n in enumerate(chunk):
        past = cached[b]
        slot = torch.arange(past + n, device=DEV)
        ids = s["table"][b][slot // page].long()
        position = slot.clone()
        above = None
        if parents:
            position[past:] = past + torch.tensor(_depths(parents[b]), device=DEV)
            above = torch.eye(n, dtype=torch.bool)
            for j in range(1, n):
                above[j] |= above[parents[b][j - 1]]
            above = above.to(DEV)
        for h in range(case["hkv"]):
            k = s["k_cache"][0, ids, slot % page, h].double()
            v = s["v_cache"][0, ids, slot % page, h].double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][0, h].double(), v * s["v_scale"][0, h].double()
            for t0 in range(0, n, 256):
                t1 = min(n, t0 + 256)
                mine = position[past + t0:past + t1, None]
                if above is None:
                    ok = slot[None] <= mine
                else:
                    ok = torch.cat((torch.ones((t1 - t0, past), dtype=torch.bool, device=DEV), above[t0:t1]), 1)
                if prefixes:
                    ok = ok | (slot[None] < prefixes[b])
                if case["window"]:
                    ok = ok & (position[None] > mine - case["window"])
                for g in range(h * G, (h + 1) * G):
                    z = (s["q"][row + t0:row + t1, g].double() @ k.T) * s["scale"]
                    if case["cap"]:
                        z = case["cap"] * torch.tanh(z / case["cap"])
                    if s["slopes"] is not None:
                        z -= s["slopes"][g].double() * (mine - position[None]).abs()
                    z = torch.where(ok, z, -math.inf)
                    l = torch.logsumexp(z, 1)
                    lse[row + t0:row + t1, g] = l
                    out[row + t0:row + t1, g] = (z - l[:, None]).exp() @ v
        row += n
    return out, lse
