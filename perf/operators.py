"""Cases of the cache operators: append, attend and compact of a paged key/value cache.

One verify step of a target model touches its cache three times. The chunk's keys and values are rotated and
appended (the last committed token and the drafts after it), the chunk attends over the cache, and once the
drafts are verified the accepted path of a token tree is moved to the front of the chunk's slots. The same
three calls serve plain decoding (chunks of one token) and prompts (long chunks).

A chunk uses the layout of the verify step: sequence b owns the rows seq_offsets[b] + b ..
seq_offsets[b + 1] + b, one more than its drafts. Row j of it goes to cache slot cached[b] + j.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "e4m3": 1}


# ----------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------
def _case(name, op, B, chunk, chunk_min, ctx, ctx_min, hq, hkv, d, page, kind="bf16", cache="bf16", order="token",
          tree=False, window=0, rot=0, interleaved=False, layers=1, lens=1):
    """chunk, ctx: largest tokens of a chunk and largest cached length (the smallest are *_min; lengths in
    between are spread evenly over the logarithm). order: "token" keeps a page as [page, head, dim] rows, "head"
    as [head, page, dim]. rot: rotated dimensions. lens: seed of the lengths."""
    return dict(name=name, op=op, B=B, chunk=chunk, chunk_min=chunk_min, ctx=ctx, ctx_min=ctx_min, hq=hq, hkv=hkv,
                d=d, page=page, kind=kind, cache=cache, order=order, tree=tree, window=window, rot=rot,
                interleaved=interleaved, layers=layers, lens=lens)


def listed():
    return [
        # plain decoding of one stream: the call's latency
        _case("append one token", "append", 1, 1, 1, 900, 900, 32, 8, 128, 16, rot=128),
        # the verify batch of the benchmark (64 sequences, 5 drafts) with an 8-bit cache
        _case("append verify 64x6 e4m3", "append", 64, 6, 6, 4000, 100, 32, 8, 128, 32, cache="e4m3", rot=128),
        # prompt chunks of a prefill batch: ragged, partly rotated interleaved heads of 96
        _case("append prompts 8 to 2048", "append", 8, 2048, 37, 5000, 1, 40, 10, 96, 64, kind="fp16", cache="fp16",
              order="head", rot=64, interleaved=True),
        # plain decoding of one stream
        _case("attend one token", "attend", 1, 1, 1, 900, 900, 32, 8, 128, 16),
        # the verify batch of the benchmark over ragged contexts
        _case("attend verify 64x6", "attend", 64, 6, 6, 8000, 500, 32, 8, 128, 16),
        # token trees of the largest size, odd heads per group
        _case("attend trees 16x32", "attend", 16, 32, 32, 4001, 300, 28, 4, 128, 32, kind="fp16", cache="fp16",
              order="head", tree=True),
        # few sequences over a long context: the work is split along it
        _case("attend long 2x8", "attend", 2, 8, 8, 131072, 60001, 64, 8, 128, 64),
        # a decoding batch of a local-attention layer without shared heads
        _case("attend window 128x1", "attend", 128, 1, 1, 6000, 1, 16, 16, 64, 32, kind="fp16", cache="fp16",
              window=1024),
        # an 8-bit cache halves the bytes of a verify batch
        _case("attend e4m3 32x4", "attend", 32, 4, 4, 16384, 2000, 32, 8, 128, 32, cache="e4m3", order="head"),
        # chunks of long prompts: bound by the matrix products
        _case("attend prompts 3x2048", "attend", 3, 2048, 700, 8192, 1, 32, 8, 128, 64),
        # one tree after its verification, a model of 4 layers
        _case("compact one tree", "compact", 1, 32, 32, 900, 900, 32, 8, 128, 16, tree=True, layers=4),
        # a verify batch of trees, 24 layers
        _case("compact trees 64x32", "compact", 64, 32, 32, 200, 10, 32, 8, 128, 32, tree=True, layers=24),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "compact"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    kind = rng.choice(["bf16", "bf16", "fp16"])
    c = dict(op=op, hq=hq, hkv=hkv, kind=kind, cache=rng.choice([kind, kind, "e4m3"]) if kind == "bf16" else kind,
             d=rng.choice([64, 128, 128, 80, 96]), page=rng.choice([8, 16, 32, 48, 64, 128]),
             order=rng.choice(["token", "head"]), tree=False, window=0, rot=0, interleaved=False, layers=1,
             lens=rng.randrange(1 << 20))
    if op == "append":
        rows = _between(rng, 1, 8000)
        c["B"] = min(rows, _between(rng, 1, 128))
        c["chunk"] = max(1, rows // c["B"])
        c["chunk_min"] = _between(rng, 1, c["chunk"])
        c["ctx"] = _between(rng, 1, 4000)
        c["ctx_min"] = _between(rng, 1, c["ctx"])
        c["tree"] = c["chunk"] <= 32 and rng.random() < 0.3
        c["rot"] = rng.choice([c["d"], 32, 64])
        c["interleaved"] = rng.random() < 0.3
    elif op == "attend":
        shape = rng.choice(["tokens", "drafts", "drafts", "trees", "prompts"])
        if shape == "prompts":
            c["chunk"] = _between(rng, 33, 2048)
            c["B"] = _between(rng, 1, 3)
            c["ctx"] = _between(rng, 1, 8192)
        else:
            c["chunk"] = 1 if shape == "tokens" else rng.randrange(2, 33)
            c["B"] = _between(rng, 1, 64)
            c["ctx"] = min(131072, _between(rng, 1, 300000 // c["B"]))
        c["chunk_min"] = _between(rng, 1, c["chunk"])
        c["ctx_min"] = _between(rng, 1, c["ctx"])
        c["tree"] = shape == "trees"
        c["window"] = rng.choice([0, 0, 0, _between(rng, 16, 4096)])
    else:
        c["B"] = _between(rng, 1, 64)
        c["chunk"] = rng.randrange(2, 33)
        c["chunk_min"] = _between(rng, 1, c["chunk"])
        c["ctx"] = _between(rng, 1, 200)
        c["ctx_min"] = _between(rng, 1, c["ctx"])
        c["tree"] = True
        c["layers"] = _between(rng, 1, 24)
    return c


# ----------------------------------------------------------------------------------------------------------
# what the lengths of a case are
# ----------------------------------------------------------------------------------------------------------
def _lengths(case):
    """(chunk lengths, cached lengths, accepted counts, parents of each sequence's drafts, accepted paths)."""
    rng = random.Random(case["lens"])
    B = case["B"]
    chunk = [_between(rng, case["chunk_min"], case["chunk"]) for _ in range(B)]
    cached = [_between(rng, case["ctx_min"], case["ctx"]) for _ in range(B)]
    chunk[0], cached[-1] = case["chunk"], case["ctx"]  # the largest are there
    parents, paths = [], []
    for n in chunk:
        par = [max(0, rng.randrange(j) - rng.randrange(3)) for j in range(1, n)] if case["tree"] else list(range(n - 1))
        node, path = 0, []
        while case["op"] == "compact":  # a walk down the tree that ends early one time in four
            below = [j for j in range(node + 1, n) if par[j - 1] == node]
            if not below or rng.random() < 0.25:
                break
            node = rng.choice(below)
            path.append(node)
        parents.append(par)
        paths.append(path)
    return chunk, cached, [len(p) for p in paths], parents, paths


def _depths(par):
    dep = [0]
    for p in par:
        dep.append(dep[p] + 1)
    return dep


def work(case):
    chunk, cached, acc, parents, _ = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    a, c = SIZE[case["kind"]], SIZE[case["cache"]]
    rows = sum(chunk)
    if case["op"] == "append":
        # q, k, v in; q out in their type, k, v out in the cache's; the table's rows, the lengths
        return {"bytes": rows * d * ((2 * hq + 2 * hkv) * a + 2 * hkv * c) + rows * case["rot"] * 4 + 12 * case["B"],
                "flops": 3 * rows * (hq + hkv) * case["rot"]}
    if case["op"] == "compact":
        moved = sum(sum(p != j + 1 for j, p in enumerate(path)) for path in _lengths(case)[4])
        return {"bytes": 4 * moved * hkv * d * c * case["layers"] + 16 * case["B"] + 4 * sum(acc), "flops": 0}
    seen = tokens = 0
    w = case["window"] or 1 << 30
    for n, past, par in zip(chunk, cached, parents):
        dep = _depths(par) if case["tree"] else range(n)
        seen += sum(min(past, max(0, w - 1 - t)) + min(w, t + 1) for t in dep)
        tokens += min(past, w - 1) + n
    return {"bytes": 2 * tokens * hkv * d * c + rows * hq * (2 * d * a + 4) + 4 * (tokens // case["page"]),
            "flops": 4 * seen * hq * d}


# ----------------------------------------------------------------------------------------------------------
# what a program has before the call
# ----------------------------------------------------------------------------------------------------------
def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    chunk, cached, acc, parents, paths = _lengths(case)
    B, hq, hkv, d, page, L = (case[k] for k in ("B", "hq", "hkv", "d", "page", "layers"))
    kind, held = TYPES[case["kind"]], TYPES[case["cache"]]
    rows = sum(chunk)
    need = [-(-(n + past) // page) for n, past in zip(chunk, cached)]
    pages, width = sum(need) + 3, max(need) + 1
    # the pages of a sequence lie anywhere in the pool
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    pool = (L, pages, page, hkv, d) if case["order"] == "token" else (L, pages, hkv, page, d)

    def cache():
        x = torch.empty(pool, dtype=held, device=DEV)
        for l in range(L):
            y = torch.randn(pool[1:], generator=g, device=DEV, dtype=torch.float16)
            x[l] = (y * 60.0).to(held) if case["cache"] == "e4m3" else y.to(held)
        return x if case["order"] == "token" else x.transpose(2, 3)

    s = dict(case=case, k_cache=cache(), v_cache=cache(), table=table)
    s["k_scale"] = s["v_scale"] = None
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.012 + 0.008 * torch.rand((L, hkv), generator=g, device=DEV)
        s["v_scale"] = 0.012 + 0.008 * torch.rand((L, hkv), generator=g, device=DEV)
    ints = dict(dtype=torch.int32, device=DEV)
    offs = [0]
    for n in chunk:
        offs.append(offs[-1] + n - 1)
    s["offs"] = torch.tensor(offs, **ints)
    s["cached"] = torch.tensor(cached, **ints)
    s["parents"] = torch.tensor(sum(parents, []) or [0], **ints) if case["tree"] else None
    s["rows"], s["most"], s["longest"] = rows, case["chunk"], max(n + past for n, past in zip(chunk, cached))
    # one projection's output: the heads of q, k and v side by side
    qkv = torch.randn((rows, (hq + 2 * hkv) * d), generator=g, device=DEV)
    qkv[:, :hq * d] *= 2.0
    qkv = qkv.to(kind)
    s["q"] = qkv[:, :hq * d].view(rows, hq, d)
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(rows, hkv, d)
    s["v"] = qkv[:, (hq + hkv) * d:].view(rows, hkv, d)
    s["scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "append":
        rot, positions = case["rot"], s["longest"]
        freq = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        angle = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * freq
        s["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()
    if case["op"] == "compact":
        s["accepted"] = torch.tensor(acc, **ints)
        flat = []
        for n, path in zip(chunk, paths):
            flat += path + [-1] * (n - 1 - len(path))
        s["path"] = torch.tensor(flat or [0], **ints)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the program's handles: the cache's description and workspace, the chunk's, the outputs' buffers
        from speculative_decoding_verification_35_gb300 import speccache as sc
        s["cache"] = sc.PagedCache(s["k_cache"], s["v_cache"], s["table"], s["k_scale"], s["v_scale"])
        s["chunk"] = sc.Chunk(s["offs"], s["cached"], s["rows"], s["most"] - 1, s["parents"])
        if case["op"] == "append":
            s["turn"] = sc.Rope(s["rope"], case["interleaved"])
            s["q_out"] = torch.empty((s["rows"], case["hq"], case["d"]), dtype=TYPES[case["kind"]], device=DEV)
        elif case["op"] == "attend":
            s["out"] = torch.empty((s["rows"], case["hq"], case["d"]), dtype=TYPES[case["kind"]], device=DEV)
            s["lse"] = torch.empty((s["rows"], case["hq"]), device=DEV)
        else:
            s["now"] = torch.empty_like(s["cached"])
    return s


# ----------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------
def _done(rc):
    if rc != 0:
        raise RuntimeError("status %d" % rc)


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "append":
            _done(s["cache"].append(s["chunk"], s["q"], s["k"], s["v"], s["q_out"], rope=s["turn"]))
            return s["k_cache"][0], s["v_cache"][0], s["q_out"]
        if op == "attend":
            _done(s["cache"].attend(s["chunk"], s["q"], s["out"], s["lse"], scale=s["scale"],
                                    window=s["case"]["window"]))
            return s["out"], s["lse"]
        _done(s["cache"].compact(s["chunk"], s["accepted"], s["path"], s["now"]))
        return s["k_cache"], s["v_cache"], s["now"]
    return {"append": _append, "attend": _attend, "compact": _compact}[op](s)


def _rows(s):
    """Per chunk token of a padded [B, most] batch: its row, and whether it is one."""
    j = torch.arange(s["most"], device=DEV)
    first = s["offs"][:-1] + torch.arange(s["case"]["B"], device=DEV)
    n = s["offs"][1:] - s["offs"][:-1] + 1
    return (first[:, None] + j).clamp(max=s["rows"] - 1), j < n[:, None]


def _lineage(s):
    """[B, most, most]: token i is j itself or above it."""
    B, n = s["case"]["B"], s["most"]
    if s["parents"] is None:
        return torch.ones((n, n), dtype=torch.bool, device=DEV).tril().expand(B, n, n)
    j = torch.arange(1, n, device=DEV)
    slot = (s["offs"][:-1, None] + j - 1).clamp(max=s["parents"].numel() - 1)
    up = torch.zeros((B, n, n), device=DEV)
    up[:, 1:] = torch.nn.functional.one_hot(s["parents"][slot].long().clamp(0, n - 1), n)
    return torch.linalg.matrix_power(up + torch.eye(n, device=DEV), 32) > 0


def _bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _to_cache(s, x, scale):
    if scale is None:
        return x.to(TYPES[s["case"]["cache"]])
    return (x / scale[0][:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _append(s):
    c = s["case"]
    rot = c["rot"]
    # each row's sequence and place in it
    starts = s["offs"][:-1] + torch.arange(c["B"], device=DEV)
    row = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(starts, row, right=True) - 1
    j = row - starts[b]
    depth = j if s["parents"] is None else (_lineage(s).sum(2) - 1)[b, j]
    cs = s["rope"][(s["cached"][b] + depth).long()]
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]

    def turned(x):
        x = x.float()
        if c["interleaved"]:
            u, w = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack((u * cos - w * sin, w * cos + u * sin), -1).flatten(-2)
        else:
            u, w = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat((u * cos - w * sin, w * cos + u * sin), -1)
        return torch.cat((y, x[..., rot:]), -1)

    slot = s["cached"][b] + j
    page = s["table"][b, slot // c["page"]].long()
    at = (slot % c["page"]).long()
    _bits(s["k_cache"])[0, page, at] = _bits(_to_cache(s, turned(s["k"]), s["k_scale"]))
    _bits(s["v_cache"])[0, page, at] = _bits(_to_cache(s, s["v"].float(), s["v_scale"]))
    return s["k_cache"][0], s["v_cache"][0], turned(s["q"]).to(s["q"].dtype)


def _attend(s):
    c = s["case"]
    B, n, L, hkv, d = c["B"], s["most"], s["longest"], c["hkv"], c["d"]
    G = c["hq"] // hkv
    row, real = _rows(s)
    slot = torch.arange(L, device=DEV)
    page = s["table"][:, slot // c["page"]].clamp(min=0).long()

    def held(x, scale):
        x = _bits(x[0])[page, slot % c["page"]].view(x.dtype).float()
        x = x if scale is None else x * scale[0][:, None]
        return x.permute(0, 2, 1, 3)  # [B, hkv, L, d]

    q = s["q"][row].float().view(B, n, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * G, d)
    score = (q @ held(s["k_cache"], s["k_scale"]).transpose(2, 3)).mul_(s["scale"])
    above = _lineage(s)
    depth = above.sum(2) - 1  # [B, n]
    past = s["cached"][:, None, None]
    i = slot - past  # place in the chunk
    new = (i >= 0) & torch.gather(above, 2, i.clamp(0, n - 1).expand(B, n, L))
    new = new & (i < n)
    old = (i < 0).expand(B, n, L)
    pos = torch.where(i < 0, slot, past + torch.gather(depth[:, None, :], 2, i.clamp(0, n - 1)))
    seen = old | new
    if c["window"]:
        seen = seen & (past + depth[:, :, None] - pos < c["window"])
    seen = seen[:, None, :, None, :].expand(B, 1, n, G, L).reshape(B, 1, n * G, L)
    score = score.masked_fill_(~seen, float("-inf"))
    top = score.amax(3, keepdim=True)
    e = score.sub_(top).exp_()
    total = e.sum(3, keepdim=True)
    out = (e @ held(s["v_cache"], s["v_scale"])) / total
    lse = total.log() + top

    def packed(x):  # [B, hkv, n * G, x] to the chunk's rows
        x = x.view(B, hkv, n, G, -1).permute(0, 2, 1, 3, 4).reshape(B, n, c["hq"], -1)
        y = torch.empty((s["rows"] + 1, *x.shape[2:]), device=DEV)
        y[torch.where(real, row, s["rows"])] = x
        return y[:s["rows"]]

    return packed(out).to(s["q"].dtype), packed(lse)[..., 0]


def _compact(s):
    c = s["case"]
    j = torch.arange(c["chunk"] - 1, device=DEV)
    offs, cached = s["offs"], s["cached"]
    moves = j < s["accepted"][:, None]
    node = s["path"][(offs[:-1, None] + j).clamp(max=s["path"].numel() - 1)]
    to = torch.where(j < (offs[1:] - offs[:-1])[:, None], j + 1, 0)  # what does not move stays where it is
    src = cached[:, None] + torch.where(moves, node, to)
    dst = cached[:, None] + to
    b = torch.arange(c["B"], device=DEV)[:, None]

    def place(slot):
        return s["table"][b, slot // c["page"]].long(), (slot % c["page"]).long()

    ps, as_ = place(src)
    pd, ad = place(dst)
    k, v = _bits(s["k_cache"]), _bits(s["v_cache"])
    k[:, pd, ad] = k[:, ps, as_]
    v[:, pd, ad] = v[:, ps, as_]
    return s["k_cache"], s["v_cache"], cached + s["accepted"] + 1


# ----------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    chunk, cached, acc, parents, paths = _lengths(case)
    return {"append": _exact_append, "attend": _exact_attend, "compact": _exact_compact}[case["op"]](
        s, case, chunk, cached, parents, paths)


def _slots(s, case, b, first, last):
    """The places (pages, offsets) of a sequence's slots first .. last - 1."""
    t = torch.arange(first, last, device=DEV)
    return s["table"][b].long()[t // case["page"]], t % case["page"]


def _exact_append(s, case, chunk, cached, parents, paths):
    h = case["rot"] // 2
    k, v = s["k_cache"][0].double(), s["v_cache"][0].double()
    q = s["q"].double()
    freq = torch.tensor([500000.0 ** (-2.0 * i / case["rot"]) for i in range(h)], dtype=torch.float64, device=DEV)
    r = 0
    for b, (n, past, par) in enumerate(zip(chunk, cached, parents)):
        dep = torch.tensor(_depths(par), dtype=torch.float64, device=DEV)
        a = torch.polar(torch.ones((n, h), dtype=torch.float64, device=DEV), (past + dep)[:, None] * freq)[:, None]

        def turn(x):  # pairs as complex numbers
            y = x.double().clone()
            even = slice(0, 2 * h, 2) if case["interleaved"] else slice(0, h)
            odd = slice(1, 2 * h, 2) if case["interleaved"] else slice(h, 2 * h)
            z = torch.complex(y[..., even].contiguous(), y[..., odd].contiguous()) * a
            y[..., even], y[..., odd] = z.real, z.imag
            return y

        pg, at = _slots(s, case, b, past, past + n)
        kk, vv = turn(s["k"][r:r + n]), s["v"][r:r + n].double()
        if s["k_scale"] is not None:
            kk = torch.clamp(kk / s["k_scale"][0].double()[:, None], -448, 448)
            vv = torch.clamp(vv / s["v_scale"][0].double()[:, None], -448, 448)
        k[pg, at], v[pg, at] = kk, vv
        q[r:r + n] = turn(s["q"][r:r + n])
        r += n
    return k, v, q


def _exact_attend(s, case, chunk, cached, parents, paths):
    hkv, G = case["hkv"], case["hq"] // case["hkv"]
    out = torch.zeros((s["rows"], case["hq"], case["d"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["rows"], case["hq"]), dtype=torch.float64, device=DEV)
    r = 0
    for b, (n, past, par) in enumerate(zip(chunk, cached, parents)):
        mask = torch.zeros((n, n), dtype=torch.bool)
        if case["tree"]:
            for j in range(n):
                if j:
                    mask[j] = mask[par[j - 1]]
                mask[j, j] = True
        else:
            mask = torch.ones((n, n), dtype=torch.bool).tril()
        mask = mask.to(DEV)
        dep = mask.sum(1) - 1
        pos = torch.cat((torch.arange(past, device=DEV), past + dep))
        ok = torch.cat((torch.ones((n, past), dtype=torch.bool, device=DEV), mask), 1)
        if case["window"]:
            ok &= (past + dep)[:, None] - pos < case["window"]
        pg, at = _slots(s, case, b, 0, past + n)
        for h in range(hkv):
            k, v = s["k_cache"][0][:, :, h], s["v_cache"][0][:, :, h]
            k, v = (_bits(x)[pg, at].view(x.dtype).double() for x in (k, v))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][0, h].double(), v * s["v_scale"][0, h].double()
            for g in range(h * G, h * G + G):
                z = (s["q"][r:r + n, g].double() @ k.T) / math.sqrt(case["d"])
                z[~ok] = -math.inf
                lse[r:r + n, g] = torch.logsumexp(z, 1)
                out[r:r + n, g] = torch.softmax(z, 1) @ v
        r += n
    return out, lse


def _exact_compact(s, case, chunk, cached, parents, paths):
    k, v = s["k_cache"].double(), s["v_cache"].double()
    table = s["table"].cpu()
    now = []
    for b, (past, path) in enumerate(zip(cached, paths)):
        for j, node in enumerate(path):  # a node lies after the slot it moves to, and never before a later one
            a, z = past + node, past + j + 1
            pa, pz = int(table[b, a // case["page"]]), int(table[b, z // case["page"]])
            k[:, pz, z % case["page"]] = k[:, pa, a % case["page"]]
            v[:, pz, z % case["page"]] = v[:, pa, a % case["page"]]
        now.append(past + len(path) + 1)
    return k, v, torch.tensor(now, dtype=torch.int32, device=DEV)
