"""Attention on capped, biased and prefixed scores against the fp64 oracle.

Tolerances as in test_gpu_cache.py, with what the score functions add to dz, the error of a score: the cap's tanh is within
2^-22 of itself, its arguments and product round by 2^-23 each, so 2^-21 cap bounds all three, and it never enlarges dz (its
slope is at most 1); the bias is one product of a slope's 2^-23 and a distance's 2^-24 with one sum, 2^-22 of the bias
and 2^-23 of the score.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.test_gpu_cache import CAPACITY, HALF_STEP, TYPES, Batch, f64, tree

pytestmark = pytest.mark.gpu
KINDS = [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")]


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


def alibi(hq):
    return (2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)).float()


def run(b, **kw):
    out = torch.full((b.rows, b.hq, b.D), 7.0, dtype=TYPES[b.kind], device="cuda")
    lse = torch.full((b.rows, b.hq), 7.0, device="cuda")
    if kw.get("prefix") is not None:
        kw["prefix"] = torch.tensor(kw["prefix"], dtype=torch.int32, device="cuda")
    assert b.cache.attend(b.chunk, b.q, out, lse, layer=b.layer, **kw) == 0
    torch.cuda.synchronize()
    return out, lse


def check(b, status=0, rows=None, **kw):
    out, lse = run(b, **kw)
    assert b.cache.status_bits() == status
    q = f64(b.q)[:b.rows]
    cap, slopes, prefix = kw.get("cap", 0.0), kw.get("slopes"), kw.get("prefix")
    want, wl, mean, big, floor, bias = oc.attend_scored(
        q, b.pages64(b.k, b.ks), b.pages64(b.v, b.vs), b.table_h, b.offs_h, b.parents_h, b.cached_h, kw.get("scale", b.D ** -0.5),
        kw.get("window", 0), cap, None if slopes is None else f64(slopes), prefix)
    u = HALF_STEP[b.kind]
    dz, part = big * (b.D + 8) * 2.0 ** -23, 2.0 ** -24
    if b.cachekind == "e4m3":
        part = 2.0 ** -17
        k1 = np.abs(np.nan_to_num(b.pages64(b.k, b.ks))).sum(-1).max()
        dz = dz + 2.0 ** -18 * np.abs(q).max(-1) * k1 * abs(kw.get("scale", b.D ** -0.5))
    dz = dz + 2.0 ** -21 * cap + 2.0 ** -22 * bias + 2.0 ** -23 * (big + bias)
    tol = mean * (2.02 * u + 2 * dz[..., None] + 2.0 ** -17) + part * floor
    sel = slice(None) if rows is None else rows
    got, gl, want, wl, tol, dz = f64(out)[sel], f64(lse)[sel], want[sel], wl[sel], tol[sel], dz[sel]
    assert np.isfinite(got).all()
    worst = np.abs(got - want) - tol
    assert worst.max() <= 0, (worst.max(), np.unravel_index(np.argmax(worst), got.shape))
    empty = np.isneginf(wl)
    assert np.array_equal(empty, np.isneginf(gl)) and not got[empty].any()
    d = np.abs(gl[~empty] - wl[~empty]) - (dz[~empty] + 2.0 ** -18 + 2.0 ** -22 * np.abs(wl[~empty]))
    assert d.size == 0 or d.max() <= 0, d.max()
    return out, lse


@pytest.mark.parametrize("kind,cache", KINDS)
@pytest.mark.parametrize("past", [0, 1, 127, 128, 1000])
def test_one_token(sc, past, kind, cache):
    b = Batch(sc, [1], [past], 8, 2, 64, 16, kind, cache, seed=past)
    check(b, cap=5.0)
    check(b, slopes=alibi(8))
    check(b, cap=50.0, slopes=alibi(8), window=100)


@pytest.mark.parametrize("kind,cache", KINDS)
@pytest.mark.parametrize("hq,hkv,D", [(32, 8, 128), (28, 4, 128), (5, 1, 80), (9, 3, 96), (128, 1, 64), (6, 2, 112)])
@pytest.mark.parametrize("chunks,cached", [([6, 1, 3, 2, 6], [300, 0, 130, 5, 1]), ([150, 1, 40], [0, 200, 129])])
def test_heads_and_chunks(sc, chunks, cached, hq, hkv, D, kind, cache):
    b = Batch(sc, chunks, cached, hq, hkv, D, 16, kind, cache, order="head", seed=D)
    check(b, cap=30.0)
    check(b, cap=2.0, slopes=alibi(hq), window=60)
    check(b, prefix=[c + n // 2 for n, c in zip(chunks, cached)])


@pytest.mark.parametrize("kind,cache", KINDS)
@pytest.mark.parametrize("tokens,group", [(4, 4), (17, 1), (8, 4), (8, 8), (13, 5), (32, 4), (43, 3), (256, 1)])
def test_rows_of_a_group(sc, tokens, group, kind, cache):
    """Every kernel, at and around its number of rows."""
    b = Batch(sc, [tokens, 1, max(1, tokens // 3)], [200, 131, 0], 2 * group, 2, 64, 32, kind, cache, seed=tokens)
    check(b, cap=20.0, slopes=alibi(2 * group), prefix=[100, 500, max(1, tokens // 4)])


@pytest.mark.parametrize("kind,cache", KINDS)
@pytest.mark.parametrize("window", [0, 3, 40])
@pytest.mark.parametrize("group", [1, 2, 6])
def test_trees(sc, kind, cache, window, group):
    """Distances in a tree count its levels, not its slots."""
    rng = np.random.default_rng(5)
    chunks = [32, 1, 17, 2, 31]
    par = [tree(rng, n) for n in chunks]
    b = Batch(sc, chunks, [200, 3, 120, 0, 96], 2 * group, 2, 64, 16, kind, cache, parents=par, seed=9)
    check(b, slopes=alibi(2 * group) * 4, window=window)
    check(b, cap=8.0, window=window)


@pytest.mark.parametrize("chunks", [[1, 1, 1], [5, 2, 6], [150, 300, 40]])
@pytest.mark.parametrize("window", [0, 1, 20, 129])
def test_prefixes(sc, chunks, window):
    """Of every length: none, within the cache, within the chunk, at its end and past it, below zero."""
    cached = [700, 10, 128]
    b = Batch(sc, chunks, cached, 8, 2, 64, 16, "fp16", "fp16", seed=window)
    for prefix in ([0, 0, 0], [-5, -2 ** 31, 3], [c + n for n, c in zip(chunks, cached)], [2 ** 31 - 1] * 3,
                   [c + (n + 1) // 2 for n, c in zip(chunks, cached)], [699, 11, 129], [c + n - 1 for n, c in zip(chunks, cached)]):
        check(b, prefix=prefix, window=window)


@pytest.mark.parametrize("kind,cache", KINDS)
def test_prompts_of_one_prefix_are_not_causal(sc, kind, cache):
    b = Batch(sc, [300, 515], [0, 77], 8, 2, 128, 32, kind, cache, seed=2)
    check(b, prefix=[300, 592], cap=50.0)
    check(b, prefix=[129, 400], slopes=alibi(8))


@pytest.mark.parametrize("kind,cache", KINDS)
@pytest.mark.parametrize("tokens", [2, 90])
@pytest.mark.parametrize("cap", [0.001, 0.5, 3.0, 1e6])
def test_caps_of_every_size(sc, tokens, cap, kind, cache):
    """Scores far below the cap, around it, and far above."""
    check(Batch(sc, [tokens, 1], [150, 40], 4, 2, 64, 16, kind, cache, seed=3, qscale=8.0), cap=cap)


@pytest.mark.parametrize("kind,cache", KINDS)
@pytest.mark.parametrize("tokens,group", [(6, 2), (90, 2)])
def test_scales_of_either_sign_and_slopes_of_either(sc, tokens, group, kind, cache):
    b = Batch(sc, [tokens, 3], [140, 7], 2 * group, 2, 64, 16, kind, cache, seed=4)
    slopes = torch.tensor([0.5, -0.01, 0.0, 2.0], device="cuda")
    for scale in (0.3, -0.3, 0.0):
        check(b, scale=scale, cap=4.0, slopes=slopes)


def test_infinite_scores_are_capped(sc):
    """An infinite product has the cap's score, as its tanh is one; the plain call's is NaN."""
    for tokens in (2, 100):
        b = Batch(sc, [tokens], [60], 2, 1, 64, 16, "bf16", "bf16", seed=1)
        b.q[0, 0, 0] = 3e38
        big = b.k.clone()
        at = int(b.table_h[0][10 // 16]), 10 % 16
        b.k[0, at[0], at[1], 0] = 0.0
        b.k[0, at[0], at[1], 0, 0] = 3e38
        out, lse = run(b, cap=10.0)
        assert out.isfinite().all() and lse.isfinite().all()
        b.k.copy_(big)


def test_nan_stays_in_its_rows(sc):
    for tokens in (3, 100):
        b = Batch(sc, [tokens, 2], [60, 9], 4, 2, 64, 16, "bf16", "bf16", seed=1)
        b.q[1, 3] = float("nan")
        out, lse = run(b, cap=10.0, slopes=alibi(4))
        assert out[1, 3].isnan().all() and lse[1, 3].isnan()
        keep = torch.ones(b.rows, 4, dtype=torch.bool, device="cuda")
        keep[1, 3] = False
        assert out[keep].isfinite().all() and lse[keep].isfinite().all()


@pytest.mark.parametrize("kind,cache", KINDS)
@pytest.mark.parametrize("chunks", [[6, 3], [150, 40]])
def test_nonfinite_values_reach_only_rows_that_see_them(sc, chunks, kind, cache):
    """In a chunk's own later tokens, within and past a prefix."""
    b = Batch(sc, chunks, [130, 20], 4, 2, 64, 16, kind, cache, seed=6)
    n = chunks[0]
    inside, past = n // 3, n - 1  # a token that all see, and one that only the last sees
    for t in (inside, past):
        s = 130 + t
        raw = b.v[0, int(b.table_h[0][s // 16]), s % 16, 0]
        if cache == "e4m3":
            raw.view(torch.uint8)[3] = 0x7F
        else:
            raw[3 if t == inside else 5] = float("nan")
    out, _ = run(b, prefix=[130 + inside + 1, 0], cap=20.0)
    hit = out[:n, :2]
    assert hit[..., 3].isnan().all()  # heads 0 and 1 read key head 0
    if cache != "e4m3":
        assert hit[-1, :, 5].isnan().all() and hit[:-1, :, 5].isfinite().all()
    assert out[:n, 2:].isfinite().all() and out[n:].isfinite().all()


def test_bad_pages_hold_nothing(sc):
    for chunks in ([4, 2], [140, 30]):
        b = Batch(sc, chunks, [200, 50], 4, 2, 64, 16, seed=7)
        b.table_h[0, 3] = -1
        b.table_h[1, 0] = 1 << 20
        b.table.copy_(torch.tensor(b.table_h))
        check(b, status=1 << 4, cap=20.0, slopes=alibi(4), prefix=[210, 40])


def test_failing_sequences_fail_alone(sc):
    b = Batch(sc, [3, 4, 2], [100, 50, 20], 4, 2, 64, 16, seed=7)
    b.cached[1] = 10 ** 6
    out, lse = run(b, cap=20.0, prefix=[101, 52, 21])
    assert b.cache.status_bits() == CAPACITY
    assert not out[3:7].any() and lse[3:7].isneginf().all()
    assert out[:3].any() and out[7:].any()


def test_nothing_given_is_the_plain_call(sc):
    """Scores that nothing is done to: bit for bit what spec_cache_attend gives."""
    from speculative_decoding_verification_35_gb300 import specverify as sv
    for chunks in ([3, 1], [100, 20]):
        b = Batch(sc, chunks, [300, 77], 8, 2, 128, 16, seed=8)
        want, wl = b.attend()
        for scores in (None, sc.SvScores(None, None, 0.0, 0)):
            out, lse = torch.zeros_like(want), torch.zeros_like(wl)
            rc = sc.spec_cache_attend_scored(b.cache.struct, 0, b.chunk.struct, sv.SV_BF16, 8, b.q.data_ptr(), b.q.stride(0), 128 ** -0.5, 0,
                                             scores, out.data_ptr(), lse.data_ptr(), None, b.cache.workspace.data_ptr(), b.cache.ws_bytes,
                                             None, torch.cuda.current_stream().cuda_stream)
            assert rc == 0
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(lse, wl)


def test_long_context_splits(sc):
    check(Batch(sc, [2, 1], [20011, 9000], 4, 1, 128, 64, seed=1), cap=30.0, slopes=alibi(4) / 64)
    check(Batch(sc, [8], [30000], 16, 2, 128, 64, "bf16", "e4m3", seed=2), cap=50.0)


def test_many_sequences(sc):
    rng = np.random.default_rng(3)
    chunks, cached = [int(x) for x in rng.integers(1, 4, 700)], [int(x) for x in rng.integers(0, 60, 700)]
    check(Batch(sc, chunks, cached, 2, 1, 64, 8), cap=6.0, slopes=alibi(2), prefix=[int(x) for x in rng.integers(0, 70, 700)])


def test_repeats_graphs_and_streams(sc):
    for chunks in ([5, 1, 6], [150, 90]):
        b = Batch(sc, chunks, [1000, 400, 3][:len(chunks)], 8, 2, 128, 16, seed=12)
        prefix = torch.tensor([1002, 30, 5][:len(chunks)], dtype=torch.int32, device="cuda")
        kw = dict(cap=25.0, slopes=alibi(8), prefix=prefix)
        first = torch.empty((b.rows, 8, 128), dtype=torch.bfloat16, device="cuda")
        assert b.cache.attend(b.chunk, b.q, first, **kw) == 0
        again = torch.empty_like(first)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        assert b.cache.attend(b.chunk, b.q, again, stream=st, **kw) == 0
        torch.cuda.synchronize()
        assert torch.equal(first, again)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            assert b.cache.attend(b.chunk, b.q, again, **kw) == 0
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, again)
        prefix += 1  # what the graph reads is the tensor's present contents
        graph.replay()
        assert b.cache.attend(b.chunk, b.q, first, **kw) == 0
        torch.cuda.synchronize()
        assert torch.equal(first, again)


@pytest.mark.parametrize("B,tokens,group", [(140, 1, 4), (60, 40, 4)])
def test_waits_that_run_out(sc, B, tokens, group):
    """With a limit of one poll some wait gives up; the launch ends and says so, and the next one is right."""
    from speculative_decoding_verification_35_gb300 import specverify as sv
    b = Batch(sc, [tokens] * B, [1500] * B, 8 * group, 8, 128, 32)
    want, wl = run(b, cap=20.0)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    scores, debug, c = sc.SvScores(None, None, 20.0, 0), sv.SvDebug(), b.cache
    debug.spin_limit = 1
    for _ in range(3):
        assert sc.spec_cache_attend_scored(c.struct, 0, b.chunk.struct, sv.SV_BF16, b.hq, b.q.data_ptr(), b.q.stride(0), b.D ** -0.5, 0, scores,
                                           out.data_ptr(), lse.data_ptr(), c.status.data_ptr(), c.workspace.data_ptr(), c.ws_bytes, debug,
                                           torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert c.status_bits() == 1 << 7
        c.status.zero_()
        again, al = run(b, cap=20.0)
        assert c.status_bits() == 0 and torch.equal(again, want) and torch.equal(al, wl)
