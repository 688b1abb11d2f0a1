"""What PagePool.reserve hands to the library (CPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import _build
    _build.build()
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_calls_do_not_write_what_they_share(sc, monkeypatch):
    """Two threads may use a pool at once, each with outputs of its own: a call inside another changes nothing of it."""
    p = sc.PagePool(ints(3, 4), ints(20), ints(3), ints(2), 16)
    monkeypatch.setattr(sc.PagePool, "_stream", lambda self, stream: None)
    before = bytes(p.struct)
    mine, theirs, got = (ints(3), ints(2)), (ints(3), ints(2)), []

    def record(at, *rest):
        if not got:
            got.append(None)
            assert p.reserve(lengths=ints(3), out_held=theirs[0], out_state=theirs[1]) == 0
            assert p.reserve(lengths=ints(3)) == 0
            assert p.reserve(lengths=ints(3), out_state=theirs[1]) == 0
        s = sc.SvPages.from_buffer_copy(at) if isinstance(at, bytes) else sc.SvPages.from_address(at)
        got.append((s.out_held, s.out_state))
        return 0
    monkeypatch.setattr(sc.lib, "spec_cache_reserve", record)
    assert p.reserve(lengths=ints(3), out_held=mine[0], out_state=mine[1]) == 0
    a, b, h, s = (t.data_ptr() for t in (*theirs, p.held, p.state))
    assert got[1:] == [(a, b), (h, s), (h, b), (mine[0].data_ptr(), mine[1].data_ptr())]
    assert bytes(p.struct) == before


def test_a_calls_own_structure_is_the_pools(sc, monkeypatch):
    """But for the outputs, whatever the addresses."""
    p = sc.PagePool(ints(3, 4), ints(20), ints(3), ints(2), 48)
    monkeypatch.setattr(sc.PagePool, "_stream", lambda self, stream: None)
    got = []
    monkeypatch.setattr(sc.lib, "spec_cache_reserve", lambda at, *rest: got.append(sc.SvPages.from_buffer_copy(at)) or 0)
    held, state = ints(3), ints(2)
    assert p.reserve(lengths=ints(3), out_held=held, out_state=state) == 0
    for f, _ in sc.SvPages._fields_:
        want = {"out_held": held.data_ptr(), "out_state": state.data_ptr()}.get(f, getattr(p.struct, f))
        assert getattr(got[0], f) == want, f


def test_the_library_takes_it(sc):
    """Refused for what it says: that it was read."""
    p = sc.PagePool(ints(3, 4), ints(20), ints(3), ints(2), 48)
    at = bytes(sc.SvPages(*(1 << 20,) * 6, 4, 48, 20, 1))
    assert sc.lib.spec_cache_reserve(at, None, 1 << 20, 3, None, None, None) == 1  # reserved is not 0
    assert len(p._before) + 16 + len(p._behind) == len(at)
