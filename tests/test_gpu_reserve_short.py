"""A pool that runs short: the sequences that go without hold nothing new, and the others keep what is theirs."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.test_gpu_reserve import I32, check, pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


def lens(*n):
    return torch.tensor(n, **I32)


@pytest.mark.parametrize("by_chunk", [False, True])
def test_who_goes_without_writes_to_no_other(sc, by_chunk):
    """A sequence gives a page back, another takes it, and the first, which wants it again, finds none: what is then appended
    past its pages is refused."""
    page, h, d = 16, 2, 32
    p = sc.PagePool.create(2, 3, 4, page)
    k, v = (torch.zeros((1, 4, page, h, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = sc.PagedCache(k, v, p.page_table)
    for n in ((33, 16), (32, 16), (32, 17)):
        assert p.reserve(lengths=lens(*n)) == 0
    assert p.held.tolist() == [2, 2] and p.state[1].item() == 0 and p.status_bits() == 0
    g = torch.Generator("cuda").manual_seed(1)

    def rows():
        return torch.randn((2, h, d), generator=g, device="cuda").to(torch.bfloat16)
    offs = lens(0, 0, 0)
    second = sc.Chunk(lens(0, 0), lens(16), 1, 0)
    theirs = sc.PagedCache(k, v, p.page_table[1:])
    assert theirs.append(second, None, rows()[:1], rows()[:1], None) == 0
    before = k.clone(), v.clone()
    one_more = sc.Chunk(offs, lens(32, 16), 2, 0)
    assert p.reserve(**(dict(chunk=one_more) if by_chunk else dict(lengths=lens(33, 17)))) == 0
    assert p.status_bits() == 1 << 9 and p.held.tolist() == [2, 2]
    first = sc.Chunk(lens(0, 0), lens(32), 1, 0)
    mine = sc.PagedCache(k, v, p.page_table[:1])
    assert mine.append(first, None, rows()[:1], rows()[:1], None) == 0
    torch.cuda.synchronize()
    assert mine.status_bits() == 1 << 4
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])
    # with a page again, it goes on
    assert p.reserve(lengths=lens(33, 0)) == 0 and mine.append(first, None, rows()[:1], rows()[:1], None) == 0
    assert p.held.tolist() == [3, 0] and p.page_table[0].tolist() == [0, 1, p.page_table[0, 2].item()] and p.page_table[0, 2] >= 0
    place = int(p.page_table[0, 2])
    assert k[0, place, 0].any()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,width", [(1, 5), (30, 12), (513, 9), (1400, 7)])
def test_stale_entries(sc, B, width, in_place):
    """Tables full of ids that their sequences gave back once: those that a sequence wanted and did not get are -1 after the
    call, others stay."""
    rng = np.random.default_rng(B)
    held, need = rng.integers(0, width, B), rng.integers(0, width + 3, B)
    need[B // 2] = width
    held[B // 2] = 0
    pages = int(held.sum()) + 2
    table, queue, state = pool(held, width, pages, seed=B)
    stale = rng.integers(0, pages, table.shape).astype(np.int32)
    table = np.where(np.arange(width) < held[:, None], table, stale)
    check(sc, table, queue, held, state, 16, lengths=need * 16 - (need > 0), bits=1 << 9, in_place=in_place)


@pytest.mark.parametrize("state", [(-1, 3), (30, 3), (0, -1), (5, 27)])
def test_a_bad_state_gives_nothing(sc, state):
    held = np.array([4, 1, 2])
    table, queue, _ = pool(held, 8, 30, seed=3)
    table[:, 5:] = 7
    check(sc, table, queue, held, np.array(state), 16, lengths=np.array([0, 100, 9 * 16]), bits=1 << 4 | 1 << 9)


def test_twice_the_same(sc):
    """A call whose counts lie elsewhere can be made again, short or not."""
    held = np.array([2, 0, 1, 3])
    table, queue, state = pool(held, 6, 8, seed=2)
    table[:, 4:] = 3
    t = [torch.tensor(np.asarray(x), **I32) for x in (table, queue, held, state)]
    p = sc.PagePool(*t, 16)
    outs = torch.empty_like(t[2]), torch.empty_like(t[3])
    want = [16, 80, 33, 49]
    ref = oc.reserve(table, queue, held, state, want, 16)
    for _ in range(2):
        assert p.reserve(lengths=lens(*want), out_held=outs[0], out_state=outs[1]) == 0
        torch.cuda.synchronize()
        for got, w in zip((t[0], t[1], outs[0], outs[1]), ref):
            assert np.array_equal(got.cpu().numpy(), w)
