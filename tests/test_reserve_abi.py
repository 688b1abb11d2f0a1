"""spec_cache_reserve's structure, and what it and its binding refuse (CPU)."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an address, never dereferenced
I32 = torch.int32


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import _build
    _build.build()
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


def test_binding_struct_matches_the_header(sc, tmp_path):
    fields = [f for f, _ in sc.SvPages._fields_]
    c = tmp_path / "sizes.c"
    c.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "speccache.h"\nint main(void){ printf("%zu\\n", sizeof(sv_pages));' +
                 " ".join(f'printf("%zu\\n", offsetof(sv_pages, {f}));' for f in fields) + ' return 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)])
    got = list(map(int, subprocess.check_output([str(exe)]).split()))
    assert got == [ctypes.sizeof(sc.SvPages)] + [getattr(sc.SvPages, f).offset for f in fields]


def pages(sc, **kw):
    a = dict(page_table=FAKE, queue=FAKE, held=FAKE, state=FAKE, out_held=FAKE, out_state=FAKE, table_stride=10, page_size=16,
             pages=100, reserved=0)
    a.update(kw)
    return sc.SvPages(**a)


def chunk(sc, **kw):
    a = dict(seq_offsets=FAKE, cached=FAKE, parents=None, B=4, rows=24, max_gamma=5, reserved=0)
    a.update(kw)
    return sc.SvChunk(**a)


def call(sc, p, c=None, **kw):
    a = dict(lengths=None if c else FAKE, B=0 if c else 4, slot_map=None, device_status=None, cuda_stream=None)
    a.update(kw)
    return sc.spec_cache_reserve(p, c, **a)


@pytest.mark.parametrize("kw", [{f: v} for f in ("page_table", "queue", "held", "state", "out_held", "out_state") for v in (None, FAKE + 2)] +
                         [dict(table_stride=0), dict(page_size=0), dict(page_size=65537), dict(pages=0), dict(pages=-4), dict(reserved=1)])
def test_bad_pages_are_refused(sc, kw):
    assert call(sc, pages(sc, **kw)) == 1
    assert call(sc, pages(sc, **kw), chunk(sc)) == 1


def test_bad_calls_are_refused(sc):
    p = pages(sc)
    for kw in (dict(lengths=FAKE + 2), dict(lengths=None), dict(B=-1), dict(B=65537), dict(slot_map=FAKE), dict(device_status=FAKE + 1)):
        assert call(sc, p, **kw) == 1, kw
    for kw in (dict(lengths=FAKE), dict(slot_map=FAKE + 4), dict(device_status=FAKE + 2)):
        assert call(sc, p, chunk(sc), **kw) == 1, kw
    for kw in (dict(B=-1), dict(B=65537), dict(cached=None), dict(seq_offsets=FAKE + 1), dict(reserved=2)):
        assert call(sc, p, chunk(sc, **kw)) == 1, kw
    assert call(sc, None) == 1


def test_binding_checks_tensors(sc, monkeypatch):
    class Reached(Exception):
        pass

    def stop(*args):
        raise Reached
    monkeypatch.setattr(sc.lib, "spec_cache_reserve", stop)
    monkeypatch.setattr(sc.PagePool, "_stream", lambda self, stream: None)

    def ints(*shape):
        return torch.zeros(shape, dtype=I32)
    good = dict(page_table=ints(3, 4), queue=ints(20), held=ints(3), state=ints(2), page_size=16)
    for kw in (dict(page_table=ints(12)), dict(page_table=ints(3, 8)[:, ::2]), dict(held=ints(4)), dict(state=ints(3)),
               dict(queue=ints(4, 5)), dict(queue=ints(40)[::2]), dict(page_size=2 ** 31)):
        with pytest.raises(ValueError):
            sc.PagePool(**{**good, **kw})
    with pytest.raises(TypeError):
        sc.PagePool(**{**good, "held": ints(3).long()})
    p = sc.PagePool(**good)
    c = sc.Chunk(ints(3), ints(2), 5, 2)
    for kw in (dict(lengths=ints(3)), dict(lengths=ints(2)), dict(chunk=c), dict(chunk=c, slot_map=torch.zeros(5, dtype=torch.int64)),
               dict(lengths=ints(3), out_held=ints(3), out_state=ints(2))):
        with pytest.raises(Reached):
            p.reserve(**kw)
    for kw in (dict(), dict(chunk=c, lengths=ints(2)), dict(lengths=ints(4)), dict(lengths=ints(6)[::2]),
               dict(lengths=ints(3), slot_map=torch.zeros(5, dtype=torch.int64)), dict(chunk=c, slot_map=torch.zeros(4, dtype=torch.int64)),
               dict(chunk=sc.Chunk(ints(5), ints(4), 9, 2)), dict(lengths=ints(3), out_held=ints(2)), dict(lengths=ints(3), out_state=ints(3))):
        with pytest.raises(ValueError):
            p.reserve(**kw)
    for kw in (dict(lengths=ints(3).long()), dict(chunk=c, slot_map=ints(5))):
        with pytest.raises(TypeError):
            p.reserve(**kw)
    other = sc.Chunk(ints(3), ints(2), 5, 2)
    other.device = 1
    with pytest.raises(ValueError, match="chunk must be on"):
        p.reserve(chunk=other)


def test_tensors_of_the_host_are_refused(sc):
    def ints(*shape):
        return torch.zeros(shape, dtype=I32)
    with pytest.raises(ValueError, match="CUDA"):
        sc.PagePool(ints(3, 4), ints(20), ints(3), ints(2), 16).reserve(lengths=ints(3))
