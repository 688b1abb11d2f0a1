"""Pages and slots on the GPU against the oracle: whole numbers, equal."""
import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


def pool(held, width, pages, seed=0, head=None):
    """(table, queue, state): sequences that hold `held` pages, the others free; the ids in random places."""
    rng = np.random.default_rng(seed)
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(held), width), -1, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    head = int(rng.integers(pages)) if head is None else head
    queue = np.full(pages, -1, np.int32)
    queue[(head + np.arange(pages - at)) % pages] = order[at:]
    return table, queue, np.array([head, pages - at], np.int32)


def check(sc, table, queue, held, state, page, lengths=None, chunk=None, bits=0, in_place=False, rows=None):
    """Runs a call and compares it; chunk: (seq_offsets, cached). Returns the pool."""
    t = [torch.tensor(np.asarray(x), **I32) for x in (table, queue, held, state)]
    p = sc.PagePool(*t, page)
    outs = (t[2], t[3]) if in_place else (torch.full_like(t[2], -9), torch.full_like(t[3], -9))
    if chunk is None:
        want = [int(n) for n in lengths]
        rc = p.reserve(lengths=torch.tensor(lengths, **I32), out_held=outs[0], out_state=outs[1])
        slots = None
    else:
        offs, cached = chunk
        B = len(cached)
        rows = int(offs[-1]) + B if rows is None else rows
        gamma = max(0, max(int(offs[b + 1]) - int(offs[b]) for b in range(B)))
        want = []
        for b in range(B):
            r, T = oc.rows_of(offs, b)
            fine = T >= 1 and r >= 0 and r + T <= rows and T <= gamma + 1 and (b > 0 or offs[0] == 0)
            want.append((int(cached[b]) + T if cached[b] >= 0 else -1) if fine else None)
        slots = torch.full((rows,), -77, dtype=torch.int64, device="cuda")
        c = sc.Chunk(torch.tensor(np.asarray(offs), **I32), torch.tensor(np.asarray(cached), **I32), rows, gamma)
        rc = p.reserve(chunk=c, slot_map=slots, out_held=outs[0], out_state=outs[1])
    assert rc == 0
    torch.cuda.synchronize()
    rt, rq, rh, rs, without = oc.reserve(table, queue, held, state, want, page)
    assert p.status_bits() == bits, p.status_bits()
    assert np.array_equal(t[0].cpu().numpy(), rt)
    assert np.array_equal(t[1].cpu().numpy(), rq)
    n = len(want)
    assert np.array_equal(outs[0].cpu().numpy()[:n], rh[:n])
    assert np.array_equal(outs[1].cpu().numpy(), rs)
    if slots is not None:
        got, ref = slots.cpu().numpy(), np.full(len(slots), -77, np.int64)
        for b in range(n):
            if want[b] is None:
                continue
            r, T = oc.rows_of(offs, b)
            s = max(int(cached[b]), 0) + np.arange(T)
            if b in without:
                ref[r:r + T] = -1
            else:
                ids = rt[b, s // page].astype(np.int64)
                ref[r:r + T] = np.where((ids >= 0) & (ids < len(queue)), ids * page + s % page, -1)
        assert np.array_equal(got, ref)
    return p


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,most", [(1, 16, 1), (1, 8, 5000), (3, 64, 700), (64, 16, 7), (511, 16, 3), (512, 32, 90), (513, 8, 40),
                                         (1500, 16, 20), (5000, 48, 9)])
def test_chunks(sc, B, page, most, in_place):
    rng = np.random.default_rng(B + page)
    T, cached = rng.integers(1, most + 1, B), rng.integers(0, 400, B)
    held = -(-(cached + rng.choice([0, 0, page, 3 * page], B)) // page)
    offs = np.concatenate([[0], np.cumsum(T - 1)])
    need = -(-(cached + T) // page)
    width = int(max(held.max(), need.max())) + 2
    pages = int(np.maximum(held, need).sum()) + 5
    table, queue, state = pool(held, width, pages, seed=B)
    check(sc, table, queue, held, state, page, chunk=(offs, cached), in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page", [(1, 16), (40, 1), (300, 17), (700, 16), (2100, 64)])
def test_lengths(sc, B, page, in_place):
    """Sequences that end, shrink and grow; the queue is just long enough, so its end is met."""
    rng = np.random.default_rng(B)
    held = rng.integers(0, 30, B)
    lengths = rng.integers(0, 30 * page, B) * (rng.random(B) < 0.7)
    need = -(-lengths // page)
    pages = max(int(held.sum()), int(need.sum()), 1)
    table, queue, state = pool(held, 31, pages, seed=B)
    check(sc, table, queue, held, state, page, lengths=lengths, in_place=in_place)


@pytest.mark.parametrize("short", [1, 10, 200])
@pytest.mark.parametrize("B", [5, 900])
def test_too_few_pages(sc, B, short):
    rng = np.random.default_rng(short)
    held, lengths = rng.integers(0, 10, B), rng.integers(0, 160, B)
    need = -(-lengths // 16)
    pages = max(int(held.sum()), int(held.sum() + (need - held).clip(0).sum() - (held - need).clip(0).sum()) - short, 1)
    if pages >= held.sum() + (need - held).clip(0).sum() - (held - need).clip(0).sum():
        pytest.skip("enough after all")
    table, queue, state = pool(held, 12, pages, seed=B)
    check(sc, table, queue, held, state, 16, lengths=lengths, bits=1 << 9)


def test_a_step_after_the_other(sc):
    """Held, state and table carried through 30 steps of growth and rollback, all in place; every page has one owner."""
    rng = np.random.default_rng(1)
    B, page, pages = 20, 16, 150
    p = sc.PagePool.create(B, 20, pages, page)
    lengths = np.zeros(B, np.int64)
    for step in range(30):
        lengths = np.clip(lengths + rng.integers(-20, 30, B), 0, 20 * page)
        lengths[rng.random(B) < 0.05] = 0
        while (-(-lengths // page)).sum() > pages:
            lengths[rng.integers(B)] = 0
        before = [x.cpu().numpy().copy() for x in (p.page_table, p.queue, p.held, p.state)]
        assert p.reserve(lengths=torch.tensor(lengths, **I32)) == 0
        ref = oc.reserve(*before, [int(n) for n in lengths], page)
        for got, want in zip((p.page_table, p.queue, p.held, p.state), ref):
            assert np.array_equal(got.cpu().numpy(), want)
        held, table, queue = p.held.cpu().numpy(), p.page_table.cpu().numpy(), p.queue.cpu().numpy()
        head, count = p.state.tolist()
        owned = np.concatenate([table[b, :held[b]] for b in range(B)] + [queue[(head + np.arange(count)) % pages]])
        assert sorted(owned) == list(range(pages))
    assert p.status_bits() == 0


def test_findings_fail_their_sequence_alone(sc):
    held = np.array([1, 2, 40, -3, 0, 1, 2])
    table, queue, state = pool([1, 2, 3, 0, 0, 1, 2], 8, 30, seed=3)
    lengths = np.array([40, -1, 50, 20, 8 * 16 + 1, 128, 0])
    check(sc, table, queue, held, state, 16, lengths=lengths, bits=1 << 4 | 1 << 9)
    # a chunk's: rows past the end, a negative length
    offs, cached = np.array([0, 3, 3, 9, 7]), np.array([10, -4, 17, 3])
    held = np.array([1, 1, 2, 0])
    table, queue, state = pool(held, 8, 30, seed=4)
    check(sc, table, queue, held, state, 16, chunk=(offs, cached), rows=11, bits=1 << 4 | 1 << 9)


@pytest.mark.parametrize("state", [(-1, 3), (30, 3), (0, -1), (0, 31), (2 ** 31 - 1, 2 ** 31 - 1), (5, 27)])
def test_a_bad_state_moves_nothing(sc, state):
    held = np.array([4, 1])
    table, queue, _ = pool(held, 8, 30, seed=3)
    check(sc, table, queue, held, np.array(state), 16, lengths=np.array([0, 100]), bits=1 << 4)


def test_bad_pages_are_reported(sc):
    held = np.array([2, 0, 1])
    table, queue, state = pool(held, 4, 9, seed=3, head=0)
    queue[0], table[0, 1] = 9, -5
    check(sc, table, queue, held, state, 16, lengths=np.array([16, 16, 16]), bits=1 << 4)
    table[0, 0] = 100
    check(sc, table, queue, held, state, 16, chunk=(np.array([0, 1, 2, 3]), np.array([3, 0, 0])), bits=1 << 4)


def test_no_sequences(sc):
    table, queue, state = pool([2], 4, 9, seed=3)
    check(sc, table, queue, np.array([2]), state, 16, lengths=np.zeros(0, np.int64))


def test_captured(sc):
    held = np.array([1, 3, 0])
    table, queue, state = pool(held, 9, 30, seed=5)
    p = sc.PagePool(*(torch.tensor(x, **I32) for x in (table, queue, held, state)), 16)
    lengths = torch.zeros(3, **I32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert p.reserve(lengths=lengths) == 0
    ref = (table, queue, held, state)
    for want in ([20, 100, 5], [0, 0, 144], [33, 33, 33]):
        lengths.copy_(torch.tensor(want))
        graph.replay()
        ref = oc.reserve(*ref[:4], want, 16)
        for got, w in zip((p.page_table, p.queue, p.held, p.state), ref):
            assert np.array_equal(got.cpu().numpy(), w)


def test_the_cache_calls_use_the_pages(sc):
    """Append through a reserved table: the token of every row lies at its slot."""
    B, page, h, d = 5, 16, 2, 32
    p = sc.PagePool.create(B, 6, 20, page)
    pages = torch.zeros((1, 20, page, h, d), dtype=torch.bfloat16, device="cuda")
    cache = sc.PagedCache(pages, torch.zeros_like(pages), p.page_table)
    cached = torch.zeros(B, **I32)
    for T in ([3, 1, 20, 7, 16], [1, 1, 17, 2, 1]):
        offs = torch.tensor(np.concatenate([[0], np.cumsum(np.array(T) - 1)]), **I32)
        rows = sum(T)
        chunk = sc.Chunk(offs, cached, rows, max(T) - 1)
        slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        k, v = (torch.randn((rows, h, d), device="cuda").to(torch.bfloat16) for _ in range(2))
        assert p.reserve(chunk=chunk, slot_map=slots) == 0
        assert cache.append(chunk, None, k, v, None) == 0
        assert torch.equal(cache.k[0].view(-1, h, d)[slots], k) and torch.equal(cache.v[0].view(-1, h, d)[slots], v)
        cached += torch.tensor(T, **I32)
    assert p.status_bits() == 0 and cache.status_bits() == 0
    assert p.held.tolist() == [-(-x // page) for x in cached.tolist()]
