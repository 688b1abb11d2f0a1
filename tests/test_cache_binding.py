"""What the cache calls' binding refuses before the library is called (CPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import _build
    _build.build()
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


class Reached(Exception):
    pass


@pytest.fixture
def calls(sc, monkeypatch):
    """A cache of two sequences and its three calls on a chunk; Reached where the library would be called."""
    for name in ("spec_cache_append", "spec_cache_attend", "spec_cache_compact"):
        def stop(*args, name=name):
            raise Reached(name, args)
        monkeypatch.setattr(sc.lib, name, stop)
    monkeypatch.setattr(sc.PagedCache, "_stream", lambda self, stream: None)
    k = torch.zeros((1, 4, 8, 2, 16), dtype=torch.bfloat16)
    cache = sc.PagedCache(k, k.clone(), torch.zeros((2, 2), dtype=torch.int32))
    q = torch.zeros((3, 4, 16), dtype=torch.bfloat16)
    kv = torch.zeros((3, 2, 16), dtype=torch.bfloat16)

    def ints(n):
        return torch.zeros(n, dtype=torch.int32)

    def append(chunk, **kw):
        cache.append(chunk, q, kv, kv, q.clone(), **kw)

    def attend(chunk, **kw):
        cache.attend(chunk, q, q.clone(), **kw)

    def compact(chunk, accepted=None, path=None, now=None):
        cache.compact(chunk, ints(chunk.B) if accepted is None else accepted, path,
                      ints(chunk.B) if now is None else now)
    return append, attend, compact


def chunk(sc, B, **kw):
    return sc.Chunk(torch.zeros(B + 1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32), 3, 2, **kw)


def test_more_sequences_than_the_page_table_has(sc, calls):
    for call in calls:
        for B in (0, 1, 2):
            with pytest.raises(Reached):
                call(chunk(sc, B))
        for B in (3, 100):
            with pytest.raises(ValueError, match="page_table"):
                call(chunk(sc, B))


def test_compact_wants_dense_tensors(sc, calls):
    compact = calls[2]
    wide = torch.zeros((2, 2), dtype=torch.int32)
    for kw in (dict(accepted=wide[:, 0]), dict(now=wide[:, 1]), dict(path=torch.zeros(8, dtype=torch.int32)[::2])):
        with pytest.raises(ValueError, match="contiguous"):
            compact(chunk(sc, 2), **kw)
    with pytest.raises(Reached):
        compact(chunk(sc, 2), accepted=wide[0], path=torch.zeros(4, dtype=torch.int32), now=wide[1])


def test_chunks_and_rotations_of_another_device(sc, calls):
    """(One device here: the numbers stand for two.)"""
    other = chunk(sc, 2)
    other.device = 1
    for call in calls:
        with pytest.raises(ValueError, match="chunk must be on"):
            call(other)
    rope = sc.Rope(torch.zeros((8, 16)))
    with pytest.raises(Reached):
        calls[0](chunk(sc, 2), rope=rope)
    rope.device = 1
    with pytest.raises(ValueError, match="rope must be on"):
        calls[0](chunk(sc, 2), rope=rope)


def test_integers_past_32_bits(sc, calls):
    """Wrapped into the library's int32 they would be other layers, windows and sizes."""
    append, attend, _ = calls
    for call in (append, attend):
        for layer in (2 ** 31, 2 ** 32, -2 ** 32, 2 ** 63):
            with pytest.raises(ValueError, match="layer"):
                call(chunk(sc, 2), layer=layer)
    for window, passed in ((0, 0), (-1, -1), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                           (2 ** 32, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 64, 2 ** 31 - 1),
                           (-2 ** 32, -2 ** 31), (-2 ** 32 + 5, -2 ** 31)):
        with pytest.raises(Reached) as got:
            attend(chunk(sc, 2), window=window)
        assert got.value.args[1][8] == passed
    one = torch.zeros(2, dtype=torch.int32)
    for rows, most in ((2 ** 32 + 1, 0), (1, 2 ** 32), (-2 ** 32, 0), (1, 2 ** 31)):
        with pytest.raises(ValueError, match="int32"):
            sc.Chunk(one, one[:1], rows, most)
