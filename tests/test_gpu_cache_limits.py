"""The cache calls at the ends of their ranges: windows, lengths, scales, offsets and batches that are rare, on the GPU.

Tolerances are those of test_gpu_cache.py, whose batches these tests use.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.test_gpu_cache import BAD_OFFSETS, CAPACITY, TYPES, Batch, f64, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


@pytest.mark.parametrize("tokens", [9, 3])
def test_fp16_weights_at_the_bound(sc, tokens):
    """A tile of one score, then a tile of another that lies above it by as much as a reference allows: as the weights'
    arguments are rounded, 128 of them sum to a little less or a little more than 2^15."""
    rng = np.random.default_rng(tokens)
    B, hkv, G = 64, 8, 8
    b = Batch(sc, [tokens] * B, [256] * B, hkv * G, hkv, 64, 16, "fp16", seed=tokens)
    b.q.zero_()
    b.q[..., :3] = 1.0
    # multiples of 2^-14 below 1024, in three parts that fp16 holds; scores are 1/8 of them
    first = -rng.integers(256 << 14, 1008 << 14, (B, hkv))
    second = first + 90852  # 8 / log2(e), rounded down
    parts = np.zeros((B, 264 + tokens, hkv, 3))
    for lo, hi, z in ((0, 128, first), (128, 256, second)):
        whole = z >> 14
        rest = z - (whole << 14)  # 14 bits
        parts[:, lo:hi] = np.stack((whole, (rest >> 4 << 4) / 16384, (rest & 15) / 16384), -1)[:, None]
    parts[:, 256:, :, 0] = -30000.0
    slots = np.arange(256 + tokens)
    for i in range(B):
        pg = torch.tensor(b.table_h[i][slots // 16].astype(np.int64), device="cuda")
        at = torch.tensor(slots % 16, device="cuda")
        k = torch.zeros((len(slots), hkv, 64), dtype=torch.float16, device="cuda")
        k[..., :3] = torch.tensor(parts[i, :len(slots)], device="cuda")
        b.k[0, pg, at] = k
        b.v[0, pg, at] = torch.where(torch.tensor(slots, device="cuda") < 128, 1.0, 3.0).half()[:, None, None]
    b.check()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 40])
@pytest.mark.parametrize("chunks,hq", [([5, 1, 6], 8), ([150, 1, 40], 8), ([32, 9, 1], 4)])
@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("bf16", "e4m3")])
def test_windows_past_every_length(sc, chunks, hq, kind, cache, window):
    """The largest window there is, a usual way to say none, and those that no int32 holds."""
    rng = np.random.default_rng(2)
    par = [tree(rng, n) for n in chunks] if hq == 4 else None
    b = Batch(sc, chunks, [300, 10, 128], hq, 2, 64, 16, kind, cache, parents=par)
    out, lse = b.check(window)
    want, wl = b.attend(0)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("tokens,group", [(6, 2), (9, 6), (90, 2)])
@pytest.mark.parametrize("scale,ks", [(0.0, None), (0.125, 1e-20), (0.125, 0.0), (1e-30, 1e-6)])
def test_zero_queries_under_tiny_scales(sc, tokens, group, scale, ks):
    """Rows of zeros weigh every slot alike, also where the factor of their scores is next to nothing."""
    b = Batch(sc, [tokens, 1], [200, 30], 2 * group, 2, 64, 16, "bf16", "e4m3")
    if ks is not None:
        b.ks.fill_(ks)
    b.q[::2] = 0
    b.q[1, 0, 3] = 0
    out = torch.empty((b.rows, b.hq, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((b.rows, b.hq), device="cuda")
    assert b.cache.attend(b.chunk, b.q, out, lse, scale=scale) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0
    # the scores are under 1e-15 in every row
    b.q = torch.zeros_like(b.q)
    b.compare(out, lse)


@pytest.mark.parametrize("tokens,group", [(6, 2), (9, 6), (90, 2)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_scales_reach_their_heads(sc, tokens, group, which):
    b = Batch(sc, [tokens, 1], [200, 30], 2 * group, 2, 64, 16, "bf16", "e4m3")
    good, gl = b.attend()
    (b.ks if which == "k" else b.vs)[0, 1] = float("nan")
    out, lse = b.attend()
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0
    assert torch.equal(out[:, :group], good[:, :group]) and torch.equal(lse[:, :group], gl[:, :group])
    assert torch.isnan(out[:, group:]).all()
    assert torch.isnan(lse[:, group:]).all() if which == "k" else torch.equal(lse[:, group:], gl[:, group:])


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("group,B", [(1, 2), (3, 2), (5, 40), (3, 900), (11, 700)])
def test_other_sequences_queries_change_nothing(sc, group, B, kind, cache):
    """Chunks of one and of two tokens: the outputs of the first are the same to the bit whatever the others' queries."""
    chunks = [1 + i % 2 for i in range(B)]
    b = Batch(sc, chunks, [400 + i % 3 * 150 for i in range(B)], group, 1, 64, 16, kind, cache, seed=group, qscale=1.0)
    single = torch.tensor([n == 1 for n in chunks for _ in range(n)], device="cuda")
    q = b.q.clone()
    b.q = torch.where(single[:, None, None], q, q * 0.01)
    want, wl = b.attend()
    for factor in (40.0, -300.0):
        b.q = torch.where(single[:, None, None], q, q * factor)
        out, lse = b.attend()
        torch.cuda.synchronize()
        assert torch.equal(out[single], want[single]) and torch.equal(lse[single], wl[single])
    assert b.cache.status_bits() == 0


@pytest.mark.parametrize("offs,max_gamma,rows,stored", [
    ([0, 5, 3, 8], 5, 11, [0, 2]),      # a sequence that ends before it begins; row 5 is claimed by two others
    ([0, 5, 9, 8], 5, 11, [0, 1]),      # the last one does
    ([0, 3, 9, 11], 5, 14, [0, 2]),     # one drafts too many
    ([0, 2, 5, 8], 5, 10, [0, 1]),      # the last one's rows are not all there
    ([0, 9, 2, 12, 14], 9, 18, [0, 3]),  # too long a sequence after one that ends before it begins
])
def test_append_reports_every_bad_sequence(sc, offs, max_gamma, rows, stored):
    """The three calls find the same in a batch's offsets, also in sequences that own no row."""
    B = len(offs) - 1
    b = Batch(sc, [6] * B, [40] * B, 4, 2, 64, 8, poison=False)
    for name in ("q", "kn", "vn"):
        setattr(b, name, torch.randn((20, getattr(b, name).shape[1], 64), device="cuda").bfloat16())
    b.table = torch.arange(B * 8, dtype=torch.int32, device="cuda").view(B, 8)
    b.k = torch.randn((1, B * 8, 8, 2, 64), device="cuda").bfloat16()
    b.v = b.k.clone()
    b.offs = torch.tensor(offs, dtype=torch.int32, device="cuda")
    b.make(max_gamma)
    b.chunk.struct.rows = b.chunk.rows = rows
    q_out = torch.full((20, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    k0 = b.k.clone()
    assert b.cache.append(b.chunk, b.q, b.kn, b.vn, q_out) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == BAD_OFFSETS
    # a sequence's tokens, but for rows that another one claims as well
    claims = [i for s in range(B) for i in range(offs[s] + s, offs[s + 1] + s + 1)]
    for s in range(B):
        at = b.k[0, b.table[s].long()].reshape(64, 2, 64)
        was = k0[0, b.table[s].long()].reshape(64, 2, 64)
        assert torch.equal(at[:40], was[:40])
        if s not in stored:
            assert torch.equal(at, was)
            continue
        T = offs[s + 1] - offs[s] + 1
        assert torch.equal(at[40 + T:], was[40 + T:])
        for j in range(T):
            r = offs[s] + s + j
            if claims.count(r) == 1:
                assert torch.equal(at[40 + j], b.kn[r]) and torch.equal(q_out[r], b.q[r])
    for call in (lambda: b.cache.attend(b.chunk, b.q, q_out),
                 lambda: b.cache.compact(b.chunk, torch.zeros(B, dtype=torch.int32, device="cuda"), None,
                                         torch.empty_like(b.cached))):
        b.cache.status.zero_()
        assert call() == 0
        torch.cuda.synchronize()
        assert b.cache.status_bits() == BAD_OFFSETS


@pytest.mark.parametrize("in_place", [False, True])
def test_linear_compaction_of_long_chunks(sc, in_place):
    """Linear drafts have no limit: a prompt's chunk is kept whole."""
    chunks, past = [40, 300, 33, 32, 5], [10, 0, 30, 5, 6]
    b = Batch(sc, chunks, past, 2, 2, 64, 8, poison=False)
    i32 = dict(dtype=torch.int32, device="cuda")
    k0 = b.k.clone()
    now = b.cached if in_place else torch.zeros(5, **i32)
    assert b.cache.compact(b.chunk, torch.tensor([39, 299, 33, 31, -1], **i32), None, now) == 0
    torch.cuda.synchronize()
    # the third accepts more than it drafted
    assert now.tolist() == [50, 300, 30, 37, 6] and torch.equal(b.k, k0) and b.cache.status_bits() == BAD_OFFSETS


def test_offsets_past_the_last_one(sc):
    """Parents and paths end with the last sequence's: one that claims more, though its rows are there, fails."""
    offs = [0, 3, 20, 8]
    b = Batch(sc, [4, 4, 4], [20, 20, 20], 4, 2, 64, 8, poison=False)
    for name in ("q", "kn", "vn"):
        setattr(b, name, torch.randn((40, getattr(b, name).shape[1], 64), device="cuda").bfloat16())
    b.table = torch.arange(24, dtype=torch.int32, device="cuda").view(3, 8)
    b.k = torch.randn((1, 24, 8, 2, 64), device="cuda").bfloat16()
    b.v = b.k.clone()
    b.offs = torch.tensor(offs, dtype=torch.int32, device="cuda")
    b.parents = torch.zeros(64, dtype=torch.int32, device="cuda")  # more room than a batch's 8, so that any read is in it
    b.make(31)
    b.chunk.struct.rows = b.chunk.rows = 40
    k0 = b.k.clone()
    q_out = torch.full((40, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    assert b.cache.append(b.chunk, b.q, b.kn, b.vn, q_out) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == BAD_OFFSETS
    diff = (b.k != k0)[0].flatten(2).any(2).nonzero().tolist()
    assert diff == [[s // 8, s % 8] for s in range(20, 24)] and (q_out[4:] == 7).all()
    out = torch.full_like(q_out, 7.0)
    b.cache.status.zero_()
    assert b.cache.attend(b.chunk, b.q, out) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == BAD_OFFSETS and (out[4:] == 7).all() and torch.isfinite(out[:4]).all()
    k1, now = b.k.clone(), torch.zeros(3, dtype=torch.int32, device="cuda")
    path = torch.tensor([3] + [-1] * 2 + [5] + [-1] * 60, dtype=torch.int32, device="cuda")
    b.cache.status.zero_()
    assert b.cache.compact(b.chunk, torch.tensor([1, 1, 0], dtype=torch.int32, device="cuda"), path, now) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == BAD_OFFSETS and now.tolist() == [22, 20, 20]
    assert (b.k != k1)[0].flatten(2).any(2).nonzero().tolist() == [[2, 5]]


def test_lengths_next_to_32_bits(sc):
    """A sequence's slots end 128 below 2^31, so that a tile's last one is an int32: past that it is out of capacity,
    whatever the page table would hold."""
    b = Batch(sc, [2, 2], [20, 20], 4, 2, 64, 8, poison=False)
    k = torch.randn((1, 1, 65536, 2, 64), device="cuda").bfloat16()
    b.k, b.v = k, k.clone()
    b.table = torch.zeros((2, 32769), dtype=torch.int32, device="cuda")  # one page again and again
    b.cached.copy_(torch.tensor([2 ** 31 - 129, 40]))
    b.make()
    k0 = b.k.clone()
    q_out = torch.full((4, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    assert b.cache.append(b.chunk, b.q, b.kn, b.vn, q_out) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == CAPACITY and (q_out[:2] == 7).all()
    assert (b.k != k0)[0].flatten(2).any(2).nonzero().tolist() == [[0, 40], [0, 41]]
    b.cache.status.zero_()
    lse = torch.zeros((4, 4), device="cuda")
    assert b.cache.attend(b.chunk, b.q, q_out, lse) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == CAPACITY
    assert not q_out[:2].any() and (lse[:2] == -float("inf")).all() and torch.isfinite(lse[2:]).all()
    # the last slots that there are
    b.cached[0] = 2 ** 31 - 130
    b.cache.status.zero_()
    assert b.cache.append(b.chunk, b.q, b.kn, b.vn, q_out) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0
    assert torch.equal(b.k[0, 0, 65536 - 130], b.kn[0]) and torch.equal(b.k[0, 0, 65536 - 129], b.kn[1])


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("wrong", [-1, 10 ** 6])
def test_append_on_a_bad_and_a_good_page(sc, kind, cache, wrong):
    """Tokens on a bad page are not stored; the chunk's others are, and every query is rotated."""
    b = Batch(sc, [6, 3], [13, 4], 4, 2, 64, 8, kind, cache, poison=False, layers=2, layer=1)
    good = [int(p) for p in b.table_h[0]]
    b.table[0, 1] = wrong  # slots 8 to 15; the chunk has 13 to 18
    tab = torch.randn((40, 64), device="cuda")
    rope = sc.Rope(tab)
    want = torch.empty((9, 4, 64), dtype=torch.bfloat16, device="cuda")
    q_out = torch.full_like(want, 7.0)
    k0, v0 = b.k.float().clone(), b.v.float().clone()
    assert b.cache.append(b.chunk, b.q, b.kn, b.vn, q_out, rope, layer=1) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == BAD_OFFSETS
    slots = sorted([good[s // 8], s % 8] for s in range(16, 19))
    slots = sorted(slots + [[int(b.table_h[1][s // 8]), s % 8] for s in range(4, 7)])
    for x, x0 in ((b.k, k0), (b.v, v0)):
        assert torch.equal(x[0].float(), x0[0])
        assert sorted((x.float() != x0)[1].flatten(2).any(2).nonzero().tolist()) == slots
    # as on a table without the bad page
    k1, v1 = b.k.float().clone(), b.v.float().clone()
    b.table.copy_(torch.tensor(b.table_h))
    b.cache.status.zero_()
    assert b.cache.append(b.chunk, b.q, b.kn, b.vn, want, rope, layer=1) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0 and torch.equal(q_out, want)
    for x, x1 in ((b.k, k1), (b.v, v1)):
        diff = (x.float() != x1)[1].flatten(2).any(2).nonzero().tolist()
        assert sorted(diff) == sorted([good[1], s % 8] for s in range(13, 16))


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_findings_in_place(sc, in_place):
    """Paths that are none keep their sequence's length and cache, also where the lengths are written over."""
    chunks, past = [4, 4, 4, 4, 4], [10, 20, 30, 5, 6]
    b = Batch(sc, chunks, past, 2, 2, 64, 8, poison=False)
    i32 = dict(dtype=torch.int32, device="cuda")
    k0 = b.k.clone()
    b.table[3, 0] = -1
    # a path that does not increase, a node past the chunk, more accepted than drafted, a bad page, a good one
    path = torch.tensor([2, 1, -1, 4, -1, -1, 1, 2, 3, 2, 3, -1, 3, -1, -1], **i32)
    now = b.cached if in_place else torch.zeros(5, **i32)
    assert b.cache.compact(b.chunk, torch.tensor([2, 1, 4, 2, 1], **i32), path, now) == 0
    torch.cuda.synchronize()
    assert b.cache.status_bits() == BAD_OFFSETS
    assert now.tolist() == [10, 20, 30, 8, 8]
    diff = (b.k != k0)[0].flatten(2).any(2).nonzero().tolist()
    assert diff == [[int(b.table_h[4][0]), 7]]


@pytest.mark.parametrize("chunks", [[1, 1, 1, 1], [6, 2, 5, 1], [130, 60, 9, 200]])
def test_between_library_products(sc, chunks):
    """Calls right after products of the library, which hold tensor memory as well, and beside those of another stream."""
    b = Batch(sc, chunks, [2000, 700, 90, 300], 32, 8, 128, 16)
    want, wl = b.attend()
    x = torch.randn((512, 2048), device="cuda").bfloat16()
    w = torch.randn((2048, 2048), device="cuda").bfloat16() * 2048 ** -0.5
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for i in range(40):
        with torch.cuda.stream(side):
            y = x[:8 << i % 7] @ w
        z = x[:8 << i % 7] @ w
        got.append(b.attend())
        z = z @ w
        got.append(b.attend())
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0 and torch.isfinite(y).all() and torch.isfinite(z).all()
    for out, lse in got:
        assert torch.equal(out, want) and torch.equal(lse, wl)
