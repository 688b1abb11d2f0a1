"""The cache calls on the GPU against the fp64 oracle.

Tolerances, from the formulas. u is half a step of the outputs' type (2^-8 bf16, 2^-11 fp16), M the mean of |v|
under the exact weights, z the scores, S the largest sum_d |scale q_d k_d| of a row and head:
  scores     |dz| <= S (D + 8) 2^-23  (float products and sums, one step each)
             e4m3 caches: the query may be split into parts that are kept to 2^-18 of its largest element
  weights    |dw| <= w (u + 2 |dz| + 2^-18)  (their rounding to the outputs' precision, exp), and for weights far
             below the largest an absolute part: 2^-24 of the largest one (fp16), 2^-17 (e4m3 caches)
  out        |d| <= M (2.02 u + 2 |dz| + 2^-17) + that part times sum |v| / sum w
  lse        |d| <= |dz| + 2^-18 + 2^-22 |lse|
Appended keys: one rounding of x c - w s, whose float error is at most 2^-22 (|x| + |w|); e4m3 half a step 2^-4
of the value and 2^-10 where it is subnormal.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
BAD_OFFSETS, CAPACITY = 1 << 4, 1 << 9


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


def f64(t):
    return t.float().double().cpu().numpy()


class Batch:
    """A batch of chunks over a scattered paged cache, everything no token sees filled with NaN."""

    def __init__(self, sc, chunks, cached, hq, hkv, D, page, kind="bf16", cache=None, order="token", parents=None,
                 layers=1, layer=0, seed=0, spare=2, width=1, poison=True, qscale=2.0):
        self.sc, self.kind, self.cachekind = sc, kind, cache or kind
        self.chunks, self.cached_h, self.hq, self.hkv, self.D, self.page = chunks, cached, hq, hkv, D, page
        rng = np.random.default_rng(seed)
        self.rng = rng
        B = len(chunks)
        need = [-(-(t + c) // page) for t, c in zip(chunks, cached)]
        n = sum(need) + spare
        order_ = rng.permutation(n)
        self.table_h = np.full((B, max(need) + width), -1, dtype=np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table_h[b, :m] = order_[at:at + m]
            at += m
        self.offs_h = np.concatenate([[0], np.cumsum(np.array(chunks) - 1)]).astype(np.int32)
        self.rows = sum(chunks)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        held = TYPES[self.cachekind]
        shape = (layers, n, page, hkv, D) if order == "token" else (layers, n, hkv, page, D)
        mag = 60.0 if cache == "e4m3" else 1.0

        def pool():
            x = (torch.randn(shape, generator=g, device="cuda") * mag).to(held)
            return x if order == "token" else x.transpose(2, 3)
        self.k, self.v = pool(), pool()
        self.ks = self.vs = None
        if self.cachekind == "e4m3":
            self.ks = 0.012 + 0.008 * torch.rand((layers, hkv), generator=g, device="cuda")
            self.vs = 0.012 + 0.008 * torch.rand((layers, hkv), generator=g, device="cuda")
        if poison:  # every token that belongs to no sequence
            used = torch.zeros((n, page), dtype=torch.bool)
            for b in range(B):
                s = np.arange(cached[b] + chunks[b])
                used[self.table_h[b][s // page], s % page] = True
            for x in (self.k, self.v):
                raw = x.view(torch.uint8) if self.cachekind == "e4m3" else x
                raw[:, ~used.cuda()] = 0x7F if self.cachekind == "e4m3" else float("nan")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.tensor(self.table_h, **i32)
        self.offs, self.cached = torch.tensor(self.offs_h, **i32), torch.tensor(cached, **i32)
        self.parents_h = None if parents is None else np.array(sum(parents, []) + [0], dtype=np.int32)
        self.parents = None if parents is None else torch.tensor(self.parents_h, **i32)
        dt = TYPES[kind]
        qkv = torch.randn((max(self.rows, 1), (hq + 2 * hkv) * D), generator=g, device="cuda")
        qkv[:, :hq * D] *= qscale
        qkv = qkv.to(dt)
        self.q = qkv[:, :hq * D].view(-1, hq, D)
        self.kn = qkv[:, hq * D:(hq + hkv) * D].view(-1, hkv, D)
        self.vn = qkv[:, (hq + hkv) * D:].view(-1, hkv, D)
        self.layer = layer
        self.make()

    def make(self, max_gamma=None):
        sc = self.sc
        self.cache = sc.PagedCache(self.k, self.v, self.table, self.ks, self.vs)
        self.chunk = sc.Chunk(self.offs, self.cached, self.rows,
                              max(self.chunks) - 1 if max_gamma is None else max_gamma, self.parents)

    def attend(self, window=0, stream=None, lse=True):
        out = torch.full((self.rows, self.hq, self.D), 7.0, dtype=TYPES[self.kind], device="cuda")
        ls = torch.full((self.rows, self.hq), 7.0, device="cuda") if lse else None
        rc = self.cache.attend(self.chunk, self.q, out, ls, window=window, layer=self.layer, stream=stream)
        assert rc == 0, rc
        return out, ls

    def pages64(self, x, s):
        y = f64(x[self.layer])
        return y if s is None else y * f64(s[self.layer])[:, None]

    def check(self, window=0, status=0):
        out, lse = self.attend(window)
        torch.cuda.synchronize()
        assert self.cache.status_bits() == status
        self.compare(out, lse, window)
        return out, lse

    def compare(self, out, lse, window=0, rows=None):
        q = f64(self.q)[:self.rows]
        want, wl, mean, big, floor = oc.attend(q, self.pages64(self.k, self.ks), self.pages64(self.v, self.vs),
                                               self.table_h, self.offs_h, self.parents_h, self.cached_h,
                                               self.D ** -0.5, window)
        u = HALF_STEP[self.kind]
        dz = big * (self.D + 8) * 2.0 ** -23
        part = 2.0 ** -24
        if self.cachekind == "e4m3":
            part = 2.0 ** -17
            k1 = np.abs(np.nan_to_num(self.pages64(self.k, self.ks))).sum(-1).max()
            dz = dz + 2.0 ** -18 * np.abs(q).max(-1) * k1 * self.D ** -0.5
        tol = mean * (2.02 * u + 2 * dz[..., None] + 2.0 ** -17) + part * floor
        sel = slice(None) if rows is None else rows
        got, gl = f64(out)[sel], f64(lse)[sel]
        want, wl, tol, dz = want[sel], wl[sel], tol[sel], dz[sel]
        assert np.isfinite(got).all()
        worst = np.max((np.abs(got - want) - tol))
        assert worst <= 0, (worst, np.unravel_index(np.argmax(np.abs(got - want) - tol), got.shape))
        empty = np.isneginf(wl)
        assert np.array_equal(empty, np.isneginf(gl)) and not got[empty].any()
        d = np.abs(gl[~empty] - wl[~empty]) - (dz[~empty] + 2.0 ** -18 + 2.0 ** -22 * np.abs(wl[~empty]))
        assert d.size == 0 or d.max() <= 0, d.max()


def tree(rng, n):
    return [max(0, int(rng.integers(j)) - int(rng.integers(3))) for j in range(1, n)]


# ------------------------------------------------------------------------------------------------
# attend
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("past", [0, 1, 7, 127, 128, 129, 1000])
def test_one_token(sc, past, kind, cache):
    Batch(sc, [1], [past], 8, 2, 64, 16, kind, cache, seed=past).check()


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("hq,hkv,D", [(8, 8, 128), (32, 8, 128), (28, 4, 128), (5, 1, 80), (9, 3, 96), (128, 1, 64),
                                      (40, 2, 16), (6, 2, 112)])
def test_ragged_drafts_and_heads(sc, hq, hkv, D, kind, cache):
    Batch(sc, [6, 1, 3, 2, 6], [300, 0, 130, 5, 1], hq, hkv, D, 16, kind, cache, order="head", seed=D).check()


@pytest.mark.parametrize("D", [8, 24, 72, 120])
def test_head_sizes_of_eight(sc, D):
    Batch(sc, [4, 2], [131, 40], 4, 2, D, 16, seed=D).check()


@pytest.mark.parametrize("page", [8, 16, 24, 48, 64, 128, 136, 256, 1024])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_page_sizes(sc, page, cache):
    Batch(sc, [3, 5], [517, 260], 4, 2, 128, page, "bf16", cache, seed=page).check()


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("window", [0, 2, 30])
def test_trees(sc, kind, cache, window):
    rng = np.random.default_rng(5)
    chunks = [32, 1, 17, 2, 31]
    par = [tree(rng, n) for n in chunks]
    Batch(sc, chunks, [200, 3, 120, 0, 96], 12, 2, 64, 16, kind, cache, parents=par, seed=9).check(window)


@pytest.mark.parametrize("window", [1, 2, 17, 128, 129, 300, 100000])
@pytest.mark.parametrize("chunks", [[1, 1, 1], [5, 2, 6], [150, 1, 40]])
def test_windows(sc, window, chunks):
    b = Batch(sc, chunks, [700, 10, 128], 8, 2, 64, 16, "fp16", "fp16", seed=window)
    # pages wholly below every window may be gone: their table entries are not read
    for i, (n, c) in enumerate(zip(chunks, [700, 10, 128])):
        gone = max(0, c - window + 1) // 16
        b.table_h[i, :gone] = -1
    b.table.copy_(torch.tensor(b.table_h))
    b.check(window)


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("chunks,cached,hq,hkv,D", [([300, 515], [0, 77], 8, 2, 128), ([129], [1000], 3, 1, 64),
                                                    ([33, 64, 700], [1, 500, 0], 14, 2, 96)])
def test_prompts(sc, chunks, cached, hq, hkv, D, kind, cache):
    Batch(sc, chunks, cached, hq, hkv, D, 32, kind, cache, seed=sum(chunks)).check()


def test_many_sequences(sc):
    rng = np.random.default_rng(3)
    Batch(sc, [int(x) for x in rng.integers(1, 4, 700)], [int(x) for x in rng.integers(0, 60, 700)], 2, 1, 64, 8).check()


def test_layers_and_strides(sc):
    b = Batch(sc, [4, 4], [100, 20], 8, 2, 128, 16, layers=3, layer=2, cache="e4m3")
    b.check()
    # keys and values as slices of one array, [page][2][token][head][dim]
    b = Batch(sc, [4, 4], [100, 20], 8, 2, 128, 16)
    both = torch.stack((b.k, b.v), 2)
    b.k, b.v = both[:, :, 0], both[:, :, 1]
    b.make()
    b.check()


def test_long_context_splits(sc):
    Batch(sc, [2, 1], [20011, 9000], 4, 1, 128, 64, seed=1).check()
    Batch(sc, [8], [30000], 16, 2, 128, 64, "bf16", "e4m3", seed=2).check()


@pytest.mark.parametrize("value", [30.0, -30.0])
def test_large_scores(sc, value):
    """Scores whose running maximum climbs steadily along the cache, or falls."""
    b = Batch(sc, [3], [600], 4, 1, 64, 16, qscale=1.0)
    ramp = torch.linspace(0, value, 640, device="cuda")
    b.q[..., 0] = 8.0
    for s in range(603):
        b.k[0, int(b.table_h[0][s // 16]), s % 16, :, 0] = ramp[s]
    b.check()


def test_offsets_past_32_bits(sc):
    n = 140000  # pages of 16 x 8 x 128: the last ones lie past 2^31 elements
    b = Batch(sc, [2, 3], [60, 33], 8, 8, 128, 16)
    k = torch.empty((1, n, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    at = torch.tensor([n - 1 - i for i in range(b.k.shape[1])], device="cuda")
    k[:, at], v[:, at] = b.k, b.v
    small_k, small_v, small_t = b.k, b.v, b.table_h
    b.k, b.v = k, v
    b.table = torch.where(b.table >= 0, n - 1 - b.table, b.table).to(torch.int32)
    b.make()
    out, lse = b.attend()
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0
    b.k, b.v, b.table_h = small_k, small_v, small_t
    b.compare(out, lse)


def test_bad_pages_hold_nothing(sc):
    b = Batch(sc, [2, 3, 2], [60, 200, 5], 8, 2, 64, 16)
    b.table_h[0, 1] = -3
    b.table_h[1, 5] = 10 ** 6
    b.table_h[2, :] = b.k.shape[1]
    b.table.copy_(torch.tensor(b.table_h))
    b.check(status=BAD_OFFSETS)


def test_failing_sequences_fail_alone(sc):
    rng = np.random.default_rng(6)
    chunks = [3, 4, 2, 5, 3]
    par = [tree(rng, n) for n in chunks]
    b = Batch(sc, chunks, [40, 20, 30, 10, 60], 8, 2, 64, 16, parents=par)
    good, gl = b.attend()
    b.cached[1] = -1
    b.cached[2] = 5 * 16 - 1  # one token past the table
    bad = b.parents.clone()
    o = int(b.offs_h[3])
    bad[o + 2] = 3  # node 3 under itself
    b.parents.copy_(bad)
    out, lse = b.attend()
    torch.cuda.synchronize()
    assert b.cache.status_bits() == BAD_OFFSETS | CAPACITY
    r = np.cumsum([0] + chunks)
    for i, ok in enumerate([True, False, False, False, True]):
        s = slice(r[i], r[i + 1])
        if ok:
            assert torch.equal(out[s], good[s]) and torch.equal(lse[s], gl[s])
        else:
            assert not out[s].any() and (lse[s] == -float("inf")).all()


def test_bad_offsets_write_no_rows(sc):
    b = Batch(sc, [3, 4, 2], [40, 20, 30], 8, 2, 64, 16)
    good, _ = b.attend()
    b.make(max_gamma=2)  # sequence 1 has three drafts
    out, _ = b.attend()
    torch.cuda.synchronize()
    assert b.cache.status_bits() == BAD_OFFSETS
    assert torch.equal(out[:3], good[:3]) and (out[3:7] == 7).all() and torch.equal(out[7:], good[7:])
    b.make()
    b.chunk.struct.rows = 8  # the last sequence's rows are not all there
    out, _ = b.attend()
    torch.cuda.synchronize()
    assert b.cache.status_bits() == BAD_OFFSETS
    assert torch.equal(out[:7], good[:7]) and (out[7:] == 7).all()


def test_spare_rows_are_not_written(sc):
    b = Batch(sc, [3, 4], [40, 20], 8, 2, 64, 16)
    good, _ = b.attend()
    q = torch.cat((b.q, torch.full((9, 8, 64), float("nan"), dtype=b.q.dtype, device="cuda")))
    out = torch.full((16, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    chunk = sc.Chunk(b.offs, b.cached, 16, 31)
    assert b.cache.attend(chunk, q, out, None) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0
    assert torch.equal(out[:7], good) and (out[7:] == 7).all()


def test_nan_queries_stay_in_their_rows(sc):
    b = Batch(sc, [3, 4], [40, 20], 8, 2, 64, 16)
    good, gl = b.attend()
    b.q[1, 3, 5] = float("nan")
    b.q[4, 0, 0] = float("inf")
    out, lse = b.attend()
    torch.cuda.synchronize()
    bad = torch.zeros((7, 8), dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[4, 0] = True
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
    assert torch.equal(out[~bad], good[~bad]) and torch.equal(lse[~bad], gl[~bad])


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("bf16", "e4m3")])
def test_nonfinite_values_reach_only_rows_that_see_them(sc, kind, cache):
    """A branch's or a later token's NaN or infinity in the cache changes no row that does not see it."""
    rng = np.random.default_rng(8)
    par = [[0, 0, 1, 1, 2, 3], tree(rng, 3)]
    b = Batch(sc, [7, 3], [130, 20], 4, 2, 64, 16, kind, cache, parents=par)
    good, gl = b.attend()
    slot = 130 + 3  # node 3 of sequence 0: under 1, with child 6
    pg, at = int(b.table_h[0][slot // 16]), slot % 16
    for x in (b.k, b.v):
        if cache == "e4m3":
            x.view(torch.uint8)[0, pg, at, 0, 5] = 0x7F
        else:
            x[0, pg, at, 0, 5] = float("nan")
            x[0, pg, at, 1, 6] = float("inf")
    out, lse = b.attend()
    torch.cuda.synchronize()
    sees = torch.zeros(10, dtype=torch.bool)
    sees[3] = sees[6] = True
    assert torch.equal(out[~sees], good[~sees]) and torch.equal(lse[~sees], gl[~sees])
    assert torch.isnan(out[sees][:, :2]).all() and torch.isnan(lse[sees][:, :2]).all()


def test_streams_graphs_and_repeats(sc):
    b = Batch(sc, [6, 1, 3], [3000, 100, 700], 8, 2, 128, 16)
    a, al = b.attend()
    c, cl = b.attend()
    torch.cuda.synchronize()
    assert torch.equal(a, c) and torch.equal(al, cl)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        d, dl = b.attend()
    side.synchronize()
    assert torch.equal(a, d) and torch.equal(al, dl)
    out, lse = torch.zeros_like(a), torch.zeros_like(al)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert b.cache.attend(b.chunk, b.q, out, lse) == 0
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out) and torch.equal(al, lse)
    # lengths are read on the device: a replay follows them
    b.cached_h = [2900, 50, 1]
    b.cached.copy_(torch.tensor(b.cached_h))
    g.replay()
    torch.cuda.synchronize()
    b.compare(out, lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("tokens,group", [(4, 4), (17, 1), (8, 4), (33, 1), (8, 8), (13, 5), (32, 4), (43, 3), (256, 1),
                                          (65, 4), (2, 128), (3, 127)])
def test_rows_of_a_group(sc, tokens, group, kind, cache, D):
    """tokens x group rows read the same keys: 16, 32, 64, 128, 256 of them, and just past those."""
    Batch(sc, [tokens, 1, (tokens + 1) // 2], [290, 0, 127], 2 * group, 2, D, 32, kind, cache, seed=tokens).check()


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("group,window", [(1, 0), (1, 5), (2, 0), (2, 40), (4, 0), (4, 3), (8, 200)])
def test_trees_of_a_group(sc, group, window, kind, cache):
    rng = np.random.default_rng(group)
    chunks = [32, 5, 1, 17]
    par = [tree(rng, n) for n in chunks]
    Batch(sc, chunks, [250, 128, 40, 0], 2 * group, 2, 128, 16, kind, cache, parents=par, seed=group).check(window)


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("tokens,group", [(3, 2), (6, 4), (7, 8), (100, 2)])
@pytest.mark.parametrize("value", [40.0, -40.0, 300.0])
def test_moving_references(sc, value, tokens, group, kind, cache):
    """Scores that climb (or fall) along the cache past what a weight's type holds, so that a row's reference moves."""
    b = Batch(sc, [tokens], [900], 2 * group, 2, 64, 16, kind, cache, qscale=1.0)
    b.q[..., 0] = 64.0
    slots = torch.arange(900 + tokens, device="cuda")
    ramp = value / 8 * slots / 900  # times 64 / sqrt(64)
    pages = torch.tensor(b.table_h[0].astype(np.int64), device="cuda")[slots // 16]
    for h in range(2):
        x = ramp if b.ks is None else ramp / b.ks[0, h]
        b.k[0, pages, slots % 16, h, 0] = x.clamp(-448, 448).to(b.k.dtype)
    b.check()


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("tokens,group", [(6, 2), (9, 6), (90, 2)])
def test_scales_of_either_sign_and_zero(sc, tokens, group, kind, cache):
    b = Batch(sc, [tokens, 1], [200, 30], 2 * group, 2, 64, 16, kind, cache)

    def run(q, scale):
        out = torch.empty((b.rows, b.hq, b.D), dtype=TYPES[kind], device="cuda")
        lse = torch.empty((b.rows, b.hq), device="cuda")
        assert b.cache.attend(b.chunk, q, out, lse, scale=scale) == 0
        return out, lse
    for (q1, s1), (q2, s2) in (((b.q, -0.11), (-b.q, 0.11)), ((b.q, 0.0), (0 * b.q, 0.11))):
        for x, y in zip(run(q1, s1), run(q2, s2)):
            torch.cuda.synchronize()
            assert torch.equal(x, y)
    assert b.cache.status_bits() == 0
    # with a scale of zero every slot weighs the same
    want = torch.log(torch.tensor([200.0 + t + 1 for t in range(tokens)] + [31.0], device="cuda"))
    assert (run(b.q, 0.0)[1] - want[:, None]).abs().max() <= 2.0 ** -18 + 2.0 ** -22 * 6


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("tokens,group,window", [(6, 2, 0), (12, 4, 0), (12, 4, 20), (140, 2, 0), (140, 2, 150)])
def test_nonfinite_values_of_a_chain(sc, tokens, group, window, kind, cache):
    """A token's NaN changes the rows that see the token, those at or after it and within the window, and no others."""
    b = Batch(sc, [tokens], [131], 2 * group, 2, 64, 16, kind, cache)
    good, gl = b.attend(window)
    seen = []
    for slot in (131 + tokens // 2, 131 + tokens - 1) + ((112 + tokens // 2,) if window == 20 else ()):
        pg, at = int(b.table_h[0][slot // 16]), slot % 16
        if cache == "e4m3":
            b.v.view(torch.uint8)[0, pg, at, :, 9] = 0x7F
        else:
            b.v[0, pg, at, :, 9] = float("nan") if slot % 2 else float("inf")
        seen.append(slot)
    out, lse = b.attend(window)
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0 and torch.equal(lse, gl)
    pos = 131 + np.arange(tokens)
    hit = np.zeros(tokens, dtype=bool)
    for slot in seen:
        hit |= (slot <= pos) & ((window == 0) | (slot > pos - window))
    hit = torch.tensor(hit, device="cuda")
    other = torch.arange(64, device="cuda") != 9
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(out[:, :, other], good[:, :, other])
    assert not torch.isfinite(out[hit][:, :, 9]).any()


def test_many_long_chunks(sc):
    """More sequences than a launch has threads, in chunks of more rows than one query tile."""
    rng = np.random.default_rng(4)
    Batch(sc, [int(x) for x in rng.integers(60, 80, 530)], [int(x) for x in rng.integers(0, 30, 530)], 2, 1, 64, 8).check()


@pytest.mark.parametrize("tokens,group", [(4, 2), (20, 8)])
def test_wrong_trees_among_many(sc, tokens, group):
    """More trees than a launch has threads; those whose parents are none fail alone, wherever they stand."""
    rng = np.random.default_rng(tokens)
    B = 1100
    chunks = [int(x) for x in rng.integers(2, tokens + 1, B)]
    par = [tree(rng, n) for n in chunks]
    b = Batch(sc, chunks, [int(x) for x in rng.integers(0, 40, B)], 2 * group, 2, 64, 8, parents=par)
    good, gl = b.attend()
    wrong = [0, 31, 255, 256, 511, 512, 700, 1099]
    bad = b.parents_h.copy()
    for i in wrong:
        bad[int(b.offs_h[i]) + chunks[i] - 2] = chunks[i] - 1  # the last node under itself
    b.parents.copy_(torch.tensor(bad))
    out, lse = b.attend()
    torch.cuda.synchronize()
    assert b.cache.status_bits() == BAD_OFFSETS
    r = np.cumsum([0] + chunks)
    failed = torch.zeros(b.rows, dtype=torch.bool, device="cuda")
    for i in wrong:
        failed[r[i]:r[i + 1]] = True
    assert torch.equal(out[~failed], good[~failed]) and torch.equal(lse[~failed], gl[~failed])
    assert not out[failed].any() and (lse[failed] == -float("inf")).all()


def test_bad_pages_of_prompts(sc):
    b = Batch(sc, [150, 70], [60, 200], 4, 2, 64, 16, "fp16", "fp16")
    b.table_h[0, 2] = -1
    b.table_h[1, :] = b.k.shape[1] + 5
    b.table.copy_(torch.tensor(b.table_h))
    b.check(status=BAD_OFFSETS)


@pytest.mark.parametrize("chunks", [[3, 1], [130, 70]])
def test_outputs_on_16_bytes(sc, chunks):
    b = Batch(sc, chunks, [300, 20], 4, 2, 64, 16)
    good, _ = b.attend()
    room = torch.full((good.numel() + 8,), 7.0, dtype=good.dtype, device="cuda")
    out = room[8:].view(good.shape)
    assert b.cache.attend(b.chunk, b.q, out, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, good) and (room[:8] == 7).all()


def test_calls_in_a_row_on_one_workspace(sc):
    """Launches that begin while the last one ends wait for what it writes."""
    b = Batch(sc, [6, 2, 40], [2000, 300, 0], 8, 2, 128, 16)
    other = Batch(sc, [90, 1], [10, 5000], 8, 2, 128, 16, seed=7)
    want = [x.attend()[0] for x in (b, other)]
    torch.cuda.synchronize()
    other.cache.workspace, other.cache._ws = b.cache.workspace, b.cache._ws
    got = []
    for _ in range(20):
        got.append((b.attend()[0], other.attend()[0]))
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


# ------------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, False), (64, True), (96, False), (96, True)])
@pytest.mark.parametrize("shape", ["tokens", "tree", "prompt"])
def test_append(sc, kind, cache, rot, interleaved, shape):
    rng = np.random.default_rng(rot)
    chunks = {"tokens": [1, 1, 1], "tree": [32, 1, 9], "prompt": [70, 3, 200]}[shape]
    par = [tree(rng, n) for n in chunks] if shape == "tree" else None
    past = [900, 0, 31]
    b = Batch(sc, chunks, past, 6, 2, 96, 16, kind, cache, parents=par, order="head", layers=2, layer=1, poison=False)
    freq = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    ang = np.arange(1000)[:, None] * freq
    tab = torch.tensor(np.concatenate([np.cos(ang), np.sin(ang)], 1), dtype=torch.float32, device="cuda")
    rope = sc.Rope(tab, interleaved) if rot else None
    k0, v0 = b.k.float().clone(), b.v.float().clone()
    q_out = torch.empty((b.rows, 6, 96), dtype=TYPES[kind], device="cuda")
    assert b.cache.append(b.chunk, b.q, b.kn, b.vn, q_out, rope, layer=1) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0
    f = freq if rot else None
    q, k, slots, seq = oc.append(f64(b.q), f64(b.kn), None, b.offs_h, b.parents_h, past, f, interleaved)
    # the table is rounded to float: 2^-24 of either part, and the products' and the sum's rounding
    reach_q, reach_k = np.abs(f64(b.q)).max(-1, keepdims=True) * 2, np.abs(f64(b.kn)).max(-1, keepdims=True) * 2
    u = HALF_STEP[kind]
    assert (np.abs(f64(q_out) - q) <= u * np.abs(q) * 1.01 + 2.0 ** -22 * reach_q + 2.0 ** -25).all()
    pages = b.table_h[seq, slots // 16]
    for x, x0, want, reach, s in ((b.k, k0, k, reach_k, b.ks), (b.v, v0, f64(b.vn), 0 * reach_k, b.vs)):
        got = f64(x[1])[pages, slots % 16]
        if s is None:
            assert (np.abs(got - want) <= u * np.abs(want) * 1.01 + 2.0 ** -22 * reach + 2.0 ** -25).all()
        else:
            sc1 = f64(s[1])[:, None]
            want = np.clip(want / sc1, -448, 448)
            assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) * 1.01 + 2.0 ** -10 + 2.0 ** -21 * reach / sc1).all()
        # nothing else changed
        y = x.float().clone()
        y[1, torch.tensor(pages.astype(np.int64), device="cuda"), torch.tensor(slots % 16, device="cuda")] = 0
        z = x0.clone()
        z[1, torch.tensor(pages.astype(np.int64), device="cuda"), torch.tensor(slots % 16, device="cuda")] = 0
        assert torch.equal(y, z)


def test_append_in_place_without_queries_and_nan(sc):
    b = Batch(sc, [2, 3], [4, 20], 4, 2, 64, 8, "bf16", "e4m3", poison=False)
    tab = torch.randn((40, 64), device="cuda")
    rope = sc.Rope(tab)
    q = b.q.contiguous().clone()
    q2 = torch.empty_like(q)
    assert b.cache.append(b.chunk, q, b.kn, b.vn, q2, rope) == 0
    k1 = b.k.float().clone()
    assert b.cache.append(b.chunk, q, b.kn, b.vn, q, rope) == 0
    assert torch.equal(q, q2)
    assert b.cache.append(b.chunk, None, b.kn, b.vn, None, rope) == 0
    torch.cuda.synchronize()
    assert torch.equal(b.k.float(), k1)
    b.vn[0, 0, 0], b.vn[0, 0, 1], b.vn[0, 0, 2] = float("nan"), float("inf"), -1e30
    assert b.cache.append(b.chunk, None, b.kn, b.vn, None, None) == 0
    torch.cuda.synchronize()
    row = b.v.float()[0, int(b.table_h[0][0]), 4, 0]
    assert torch.isnan(row[0]) and row[1] == 448 and row[2] == -448


def test_append_findings(sc):
    rng = np.random.default_rng(1)
    chunks = [3, 4, 2, 5]
    par = [tree(rng, n) for n in chunks]
    b = Batch(sc, chunks, [40, 20, 30, 10], 4, 2, 64, 8, parents=par, poison=False)
    bad = b.parents.clone()
    bad[int(b.offs_h[3])] = 1
    b.parents.copy_(bad)
    b.cached[0] = -5
    b.table[2, 30 // 8] = b.k.shape[1]
    k0 = b.k.clone()
    q_out = torch.full((b.rows, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    assert b.cache.append(b.chunk, b.q, b.kn, b.vn, q_out, sc.Rope(torch.randn((24, 16), device="cuda"))) == 0
    torch.cuda.synchronize()
    # sequence 1: 20 + 4 positions fit the table; 2 does not; 0 and 3 are wrong
    assert b.cache.status_bits() == BAD_OFFSETS | CAPACITY
    assert (q_out[:3] == 7).all() and (q_out[3:7] != 7).any() and (q_out[7:] == 7).all()
    diff = (b.k != k0)[0].flatten(2).any(2).nonzero().tolist()
    want = sorted([int(b.table_h[1][s // 8]), s % 8] for s in range(20, 24))
    assert sorted(diff) == want
    b.cache.status.zero_()
    assert b.cache.append(b.chunk, None, b.kn, b.vn, None, None) == 0  # sequence 2's second token has a page
    torch.cuda.synchronize()
    diff = (b.k != k0)[0].flatten(2).any(2).nonzero().tolist()
    assert all(p != b.k.shape[1] for p, _ in diff) and b.cache.status_bits() == BAD_OFFSETS | CAPACITY


# ------------------------------------------------------------------------------------------------
# compact
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("cache,D,hkv,order", [("bf16", 128, 8, "token"), ("fp16", 72, 3, "head"), ("e4m3", 64, 1, "token")])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(sc, cache, D, hkv, order, in_place):
    rng = np.random.default_rng(2)
    chunks = [32, 1, 6, 20, 4, 32, 5]
    past = [100, 0, 7, 31, 8, 0, 3]
    b = Batch(sc, chunks, past, hkv, hkv, D, 8, "bf16" if cache == "e4m3" else cache, cache, order=order, layers=3,
              poison=False, parents=[list(range(n - 1)) for n in chunks])
    acc, path = [], []
    for i, n in enumerate(chunks):
        m = [31, 0, 3, 7, -1, 12, 4][i]
        p = sorted(int(x) for x in rng.choice(np.arange(1, n), size=max(m, 0), replace=False)) if m > 0 else []
        acc.append(m)
        path += p + [-1] * (n - 1 - len(p))
    i32 = dict(dtype=torch.int32, device="cuda")
    now = b.cached if in_place else torch.full((len(chunks),), -9, **i32)
    want = [oc.compact(f64(x), b.table_h, b.offs_h, past, acc, path) for x in (b.k, b.v)]
    assert b.cache.compact(b.chunk, torch.tensor(acc, **i32), torch.tensor(path, **i32), now) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0
    for x, (w, n) in zip((b.k, b.v), want):
        assert np.array_equal(f64(x), w)
        assert now.tolist() == n.tolist()


def test_compact_linear_and_findings(sc):
    chunks, past = [4, 4, 4, 4, 4], [10, 20, 30, 5, 6]
    b = Batch(sc, chunks, past, 2, 2, 64, 8, poison=False)
    i32 = dict(dtype=torch.int32, device="cuda")
    k0 = b.k.clone()
    now = torch.zeros(5, **i32)
    assert b.cache.compact(b.chunk, torch.tensor([3, 0, -1, 2, 1], **i32), None, now) == 0
    torch.cuda.synchronize()
    assert now.tolist() == [14, 21, 30, 8, 8] and torch.equal(b.k, k0) and b.cache.status_bits() == 0
    # a path that does not increase, a node past the chunk, more accepted than drafted, a bad page, a good one
    b.table[3, 0] = -1
    path = torch.tensor([2, 1, -1, 4, -1, -1, 1, 2, 3, 2, 3, -1, 3, -1, -1], **i32)
    for dst in (now,):
        assert b.cache.compact(b.chunk, torch.tensor([2, 1, 4, 2, 1], **i32), path, dst) == 0
        torch.cuda.synchronize()
        assert b.cache.status_bits() == BAD_OFFSETS
        assert dst.tolist() == [10, 20, 30, 8, 8]
        diff = (b.k != k0)[0].flatten(2).any(2).nonzero().tolist()
        assert diff == [[int(b.table_h[4][0]), 7]]


# ------------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------------
def test_a_tree_step_keeps_the_cache_of_its_path(sc):
    """Append and attend a tree, compact an accepted path, and attend the next token: as if the path had been
    decoded token by token."""
    par = [[0, 0, 1, 2, 2, 5]]
    b = Batch(sc, [7], [50], 4, 2, 64, 16, parents=par, poison=False)
    freq = 10000.0 ** (-np.arange(32) / 32)
    ang = np.arange(100)[:, None] * freq
    rope = sc.Rope(torch.tensor(np.concatenate([np.cos(ang), np.sin(ang)], 1), dtype=torch.float32, device="cuda"))
    k0, v0 = b.k.clone(), b.v.clone()
    qr = torch.empty((7, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, _ = torch.empty_like(qr), None
    assert b.cache.append(b.chunk, b.q, b.kn, b.vn, qr, rope) == 0
    assert b.cache.attend(b.chunk, qr, out) == 0
    i32 = dict(dtype=torch.int32, device="cuda")
    assert b.cache.compact(b.chunk, torch.tensor([3], **i32), torch.tensor([2, 5, 6, -1, -1, -1], **i32), b.cached) == 0
    torch.cuda.synchronize()
    assert b.cached.tolist() == [54] and b.cache.status_bits() == 0
    nodes = torch.tensor([0, 2, 5, 6], device="cuda")
    lin = Batch(sc, [4], [50], 4, 2, 64, 16, poison=False)
    lin.k, lin.v, lin.table, lin.table_h = k0, v0, b.table, b.table_h
    lin.make()
    q1 = torch.empty((4, 4, 64), dtype=torch.bfloat16, device="cuda")
    o1 = torch.empty_like(q1)
    assert lin.cache.append(lin.chunk, b.q[nodes], b.kn[nodes], b.vn[nodes], q1, rope) == 0
    assert lin.cache.attend(lin.chunk, q1, o1) == 0
    torch.cuda.synchronize()
    s = np.arange(54)
    pg, at = b.table_h[0][s // 16], s % 16
    assert torch.equal(b.k[0, pg, at], lin.k[0, pg, at]) and torch.equal(b.v[0, pg, at], lin.v[0, pg, at])
    assert torch.equal(qr[nodes], q1)
    lin.q, lin.rows = q1, 4
    lin.compare(o1, lin.attend()[1])
    lin.compare(out[nodes], lin.attend()[1])
