"""spec_cache_attend_scored's structure, and what it and its binding refuse (CPU)."""
import ctypes
import os
import subprocess

import pytest
import torch

from tests.test_cache_abi import FAKE, ROOT, cache, chunk


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import _build
    _build.build()
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


def test_binding_struct_matches_the_header(sc, tmp_path):
    fields = [f for f, _ in sc.SvScores._fields_]
    c = tmp_path / "sizes.c"
    c.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "speccache.h"\nint main(void){ printf("%zu\\n", sizeof(sv_scores));' +
                 " ".join(f'printf("%zu\\n", offsetof(sv_scores, {f}));' for f in fields) + ' return 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)])
    got = list(map(int, subprocess.check_output([str(exe)]).split()))
    assert got == [ctypes.sizeof(sc.SvScores)] + [getattr(sc.SvScores, f).offset for f in fields]


def call(sc, scores, ch=None, c=None, **kw):
    a = dict(layer=1, dtype=sc.SV_BF16, q_heads=32, q=FAKE, q_stride=32 * 128, scale=0.1, window=0, out=FAKE, lse=FAKE,
             device_status=None, workspace=FAKE, workspace_bytes=1 << 30, debug=None, cuda_stream=None)
    a.update(kw)
    return sc.spec_cache_attend_scored(c or cache(sc), a.pop("layer"), ch or chunk(sc), scores=sc.SvScores(**scores), **a)


@pytest.mark.parametrize("scores", [dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=1e-4), dict(cap=1e7),
                                    dict(slopes=FAKE + 2), dict(prefix=FAKE + 1), dict(reserved=1)])
def test_bad_scores_are_refused(sc, scores):
    assert call(sc, scores) == 1


def test_what_attend_refuses_is_refused(sc):
    good = dict(cap=30.0, slopes=FAKE, prefix=FAKE)
    assert call(sc, good, chunk(sc, parents=FAKE)) == 1  # trees have no prefix
    for kw in (dict(layer=2), dict(dtype=sc.SV_F16), dict(q_heads=12), dict(q_stride=8), dict(scale=float("nan")), dict(window=-1),
               dict(lse=FAKE + 2), dict(q=None), dict(out=FAKE + 8)):
        assert call(sc, good, **kw) == 1, kw
    assert call(sc, good, workspace_bytes=8) == 8
    assert call(sc, good, chunk(sc, B=0)) == 0 and call(sc, good, chunk(sc, rows=0)) == 0


def test_binding_checks_tensors(sc, monkeypatch):
    class Reached(Exception):
        pass

    def stop(*args):
        raise Reached(args)
    monkeypatch.setattr(sc.lib, "spec_cache_attend_scored", stop)
    monkeypatch.setattr(sc.PagedCache, "_stream", lambda self, stream: None)
    k = torch.zeros((1, 4, 8, 2, 16), dtype=torch.bfloat16)
    c = sc.PagedCache(k, k.clone(), torch.zeros((2, 2), dtype=torch.int32))
    q = torch.zeros((3, 4, 16), dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    ch = sc.Chunk(torch.zeros(3, **i32), torch.zeros(2, **i32), 3, 2)
    trees = sc.Chunk(torch.zeros(3, **i32), torch.zeros(2, **i32), 3, 2, torch.zeros(1, **i32))
    for kw in (dict(cap=5.0), dict(slopes=torch.zeros(4)), dict(prefix=torch.zeros(2, **i32))):
        with pytest.raises(Reached):
            c.attend(ch, q, q.clone(), **kw)
    for kw in (dict(slopes=torch.zeros(3)), dict(slopes=torch.zeros(8)[::2]), dict(prefix=torch.zeros(3, **i32)), dict(prefix=torch.zeros(4, **i32)[::2])):
        with pytest.raises(ValueError):
            c.attend(ch, q, q.clone(), **kw)
    for kw in (dict(slopes=torch.zeros(4).double()), dict(prefix=torch.zeros(2))):
        with pytest.raises(TypeError):
            c.attend(ch, q, q.clone(), **kw)
    with pytest.raises(ValueError):
        c.attend(trees, q, q.clone(), prefix=torch.zeros(2, **i32))
