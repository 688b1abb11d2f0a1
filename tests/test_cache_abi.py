"""The cache calls' C ABI and binding: declarations, structures and host-side refusals (CPU).

Every call here returns before any CUDA call, so the checks run without a GPU.
"""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "speccache.h")
FAKE = 1 << 20  # an address, never dereferenced


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import _build
    _build.build()
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


def test_binding_lists_every_declared_symbol(sc):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^(?:int|size_t)\s+([a-z_]+)\s*\(", src, flags=re.M)
    assert tuple(names) == sc.EXPORTS
    for n in names:
        assert hasattr(sc.lib, n)


def test_binding_structs_match_the_header(sc, tmp_path):
    structs = (("sv_cache", sc.SvCache), ("sv_chunk", sc.SvChunk), ("sv_rope", sc.SvRope))
    lines = ['printf("%d %d\\n", SV_F16, SV_E4M3);']
    for cname, py in structs:
        lines.append(f'printf("%zu\\n", sizeof({cname}));')
        lines += [f'printf("%zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    c = tmp_path / "sizes.c"
    c.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "speccache.h"\nint main(void){ ' + " ".join(lines) +
                 ' return 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(c), "-o", str(exe)])
    got = iter(map(int, subprocess.check_output([str(exe)]).split()))
    assert (next(got), next(got)) == (sc.SV_F16, sc.SV_E4M3)
    for cname, py in structs:
        assert ctypes.sizeof(py) == next(got), cname
        for f, _ in py._fields_:
            assert getattr(py, f).offset == next(got), (cname, f)


def cache(sc, **kw):
    a = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, page_table=FAKE, stride_page=16 * 8 * 128, stride_token=8 * 128,
             stride_head=128, stride_layer=100 * 16 * 8 * 128, dtype=sc.SV_BF16, layers=2, pages=100, page_size=16,
             heads=8, head_dim=128, table_stride=10, reserved=0)
    a.update(kw)
    return sc.SvCache(**a)


def chunk(sc, **kw):
    a = dict(seq_offsets=FAKE, cached=FAKE, parents=None, B=4, rows=24, max_gamma=5, reserved=0)
    a.update(kw)
    return sc.SvChunk(**a)


def rope(sc, **kw):
    a = dict(table=FAKE, positions=100, dim=128, interleaved=0, reserved=0)
    a.update(kw)
    return sc.SvRope(**a)


BAD_CACHE = [dict(k=None), dict(v=FAKE + 8), dict(page_table=None), dict(page_table=FAKE + 2), dict(dtype=0),
             dict(dtype=4), dict(layers=0), dict(pages=0), dict(page_size=0), dict(page_size=12), dict(page_size=65544),
             dict(heads=0), dict(head_dim=0), dict(head_dim=136), dict(head_dim=12), dict(table_stride=0),
             dict(stride_page=8 * 16 * 128 + 4), dict(stride_token=64), dict(stride_head=132), dict(stride_layer=-128),
             dict(k_scale=FAKE), dict(v_scale=FAKE), dict(reserved=1)]
BAD_E4M3 = [dict(dtype=3, head_dim=72), dict(dtype=3, stride_token=8 * 128 + 8), dict(dtype=3, k_scale=FAKE + 2)]
BAD_CHUNK = [dict(seq_offsets=None), dict(cached=None), dict(cached=FAKE + 1), dict(parents=FAKE + 2),
             dict(parents=FAKE, max_gamma=32), dict(B=-1), dict(rows=-1), dict(max_gamma=-1), dict(reserved=1)]


def calls(sc):
    def append(c, ch, r=None, **kw):
        a = dict(layer=1, dtype=sc.SV_BF16, q_heads=32, q=FAKE, q_stride=48 * 128, k=FAKE, v=FAKE, kv_stride=48 * 128,
                 q_out=2 * FAKE, device_status=None, cuda_stream=None)
        a.update(kw)
        return sc.spec_cache_append(c, a.pop("layer"), ch, r, **a)

    def attend(c, ch, **kw):
        a = dict(layer=1, dtype=sc.SV_BF16, q_heads=32, q=FAKE, q_stride=32 * 128, scale=0.1, window=0, out=FAKE,
                 lse=FAKE, device_status=None, workspace=FAKE, workspace_bytes=1 << 30, cuda_stream=None)
        a.update(kw)
        return sc.spec_cache_attend(c, a.pop("layer"), ch, **a)

    def compact(c, ch, **kw):
        a = dict(out_num_accepted=FAKE, out_path=FAKE, out_cached=FAKE, device_status=None, cuda_stream=None)
        a.update(kw)
        return sc.spec_cache_compact(c, ch, **a)
    return append, attend, compact


@pytest.mark.parametrize("kw", BAD_CACHE + BAD_E4M3)
def test_bad_caches_are_refused(sc, kw):
    bad, ch = cache(sc, **kw), chunk(sc)
    for call in calls(sc):
        assert call(bad, ch) == 1
    assert sc.spec_cache_workspace_size(bad) == 0


@pytest.mark.parametrize("kw", BAD_CHUNK)
def test_bad_chunks_are_refused(sc, kw):
    for call in calls(sc):
        assert call(cache(sc), chunk(sc, **kw)) == 1


def test_missing_structures_are_refused(sc):
    for call in calls(sc):
        assert call(None, chunk(sc)) == 1
        assert call(cache(sc), None) == 1


def test_append_refusals(sc):
    append, _, _ = calls(sc)
    c, ch = cache(sc), chunk(sc)
    for kw in (dict(layer=-1), dict(layer=2), dict(dtype=0), dict(dtype=sc.SV_F16), dict(dtype=sc.SV_E4M3), dict(q_heads=0),
               dict(q_stride=32 * 128 - 8), dict(q_stride=48 * 128 + 4), dict(kv_stride=8 * 128 - 8),
               dict(kv_stride=48 * 128 + 2), dict(k=None), dict(v=FAKE + 2), dict(q=FAKE + 8), dict(q_out=None),
               dict(q_out=FAKE), dict(device_status=FAKE + 2)):
        assert append(c, ch, **kw) == 1, kw
    for kw in (dict(table=None), dict(table=FAKE + 4), dict(positions=0), dict(dim=0), dict(dim=24), dict(dim=144),
               dict(reserved=1)):
        assert append(c, ch, rope(sc, **kw)) == 1, kw
    assert append(cache(sc, dtype=sc.SV_E4M3), ch, dtype=sc.SV_F16) == 1
    assert append(c, chunk(sc, B=0), rope(sc)) == 0 and append(c, chunk(sc, rows=0), rope(sc)) == 0


def test_attend_refusals(sc):
    _, attend, _ = calls(sc)
    c, ch = cache(sc), chunk(sc)
    for kw in (dict(layer=2), dict(dtype=sc.SV_F16), dict(q_heads=0), dict(q_heads=12), dict(q_heads=8 * 129),
               dict(q_stride=8), dict(q_stride=32 * 128 + 4), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(window=-1), dict(lse=FAKE + 2), dict(q=None), dict(q=FAKE + 2), dict(out=None), dict(out=FAKE + 8),
               dict(device_status=FAKE + 1)):
        assert attend(c, ch, **kw) == 1, kw
    for kw in (dict(workspace=None), dict(workspace=FAKE + 64), dict(workspace_bytes=8)):
        assert attend(c, ch, **kw) == 8, kw
    assert attend(c, chunk(sc, B=0)) == 0 and attend(c, chunk(sc, rows=0)) == 0
    assert sc.spec_cache_workspace_size(c) > 0


def test_compact_refusals(sc):
    _, _, compact = calls(sc)
    c, ch = cache(sc), chunk(sc)
    for kw in (dict(out_num_accepted=None), dict(out_cached=None), dict(out_path=FAKE + 2), dict(out_cached=FAKE + 2),
               dict(device_status=FAKE + 2)):
        assert compact(c, ch, **kw) == 1, kw
    assert compact(c, chunk(sc, max_gamma=32)) == 1
    assert compact(c, chunk(sc, B=0)) == 0


def test_tensor_checks(sc):
    import torch
    k = torch.zeros((1, 4, 8, 2, 16), dtype=torch.bfloat16)
    table = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(TypeError):
        sc.PagedCache(k.float(), k.float(), table)
    with pytest.raises(ValueError):
        sc.PagedCache(k, torch.zeros((1, 4, 2, 8, 16), dtype=torch.bfloat16).transpose(2, 3), table)
    with pytest.raises(TypeError):
        sc.PagedCache(k, k, table.long())
    with pytest.raises(ValueError):
        sc.PagedCache(k, k, table, k_scale=torch.ones((2, 1)))
    with pytest.raises(ValueError):
        sc.Chunk(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 2, 0)
    with pytest.raises(ValueError):
        sc.Rope(torch.zeros((4, 32))[:, ::2])
    c = sc.PagedCache(k, k.clone(), table)
    ch = sc.Chunk(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 2, 0)
    q = torch.zeros((2, 4, 16), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        c.attend(ch, q, q.half())
    with pytest.raises(ValueError):
        c.attend(ch, q, torch.zeros((1, 4, 16), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        c.attend(ch, q.transpose(0, 1), q)
    with pytest.raises(ValueError):
        c.append(ch, None, q, q, None)
