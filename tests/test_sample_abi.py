"""The filtered distributions' C ABI and binding: declarations, structures and host-side refusals (CPU).

Every call here returns before any CUDA call, so the checks run without a GPU.
"""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "specsample.h")
FAKE = 1 << 20  # an address, never dereferenced


@pytest.fixture(scope="module")
def ss():
    from speculative_decoding_verification_35_gb300 import _build
    _build.build()
    from speculative_decoding_verification_35_gb300 import specsample
    return specsample


def test_binding_lists_every_declared_symbol(ss):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^(?:int|size_t)\s+([a-z_]+)\s*\(", src, flags=re.M)
    assert tuple(names) == ss.EXPORTS
    for n in names:
        assert hasattr(ss.lib, n)


def test_binding_struct_matches_the_header(ss, tmp_path):
    fields = [f for f, _ in ss.SvFilter._fields_]
    c = tmp_path / "sizes.c"
    c.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "specsample.h"\nint main(void){ printf("%d %zu\\n", '
                 'SV_MAX_FILTER_V, sizeof(sv_filter));' + " ".join(f'printf("%zu\\n", offsetof(sv_filter, {f}));' for f in fields) +
                 ' return 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(c), "-o", str(exe)])
    got = list(map(int, subprocess.check_output([str(exe)]).split()))
    assert got[:2] == [ss.SV_MAX_FILTER_V, ctypes.sizeof(ss.SvFilter)]
    assert got[2:] == [getattr(ss.SvFilter, f).offset for f in fields]


@pytest.mark.parametrize("compiler,suffix", [(["gcc", "-std=c99"], "c"), (["g++", "-std=c++17"], "cpp")])
def test_a_caller_compiles(tmp_path, compiler, suffix):
    src = tmp_path / f"caller.{suffix}"
    src.write_text('#include "specsample.h"\nint step(const sv_filter* f, void* x, const float* u, int32_t* n, float* p, uint32_t* s) {\n'
                   '    int rc = spec_filter(x, SV_BF16, 4, 100, 104, f, x, 104, n, s, 0);\n'
                   '    return rc | spec_sample(x, SV_F32, 4, 100, 100, f, u, n, p, n, s, 0);\n}\n')
    subprocess.check_call(compiler + ["-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER), str(src)])


def filt(ss, **kw):
    a = dict(temperature=FAKE, top_k=FAKE, top_p=FAKE, min_p=FAKE, request=None, requests=4, reserved=0)
    a.update(kw)
    return ss.SvFilter(**a)


def calls(ss):
    common = dict(logits=FAKE, dtype=ss.SV_BF16, rows=4, V=100, stride=100, out_kept=FAKE, device_status=None, cuda_stream=None)

    def mask(f, **kw):
        return ss.spec_filter(**{**common, "out": 2 * FAKE, "out_stride": 100, "filter": f, **kw})

    def sample(f, **kw):
        return ss.spec_sample(**{**common, "uniforms": FAKE, "out_tokens": FAKE, "out_logprob": None, "filter": f, **kw})
    return mask, sample


@pytest.mark.parametrize("kw", [dict(logits=None), dict(logits=FAKE + 1), dict(dtype=2), dict(dtype=3), dict(rows=-1), dict(V=0),
                                dict(V=-3), dict(V=262145, stride=262145), dict(stride=99), dict(stride=1 << 38), dict(out_kept=FAKE + 2),
                                dict(device_status=FAKE + 1), dict(rows=5)])
def test_bad_arguments_are_refused(ss, kw):
    for call in calls(ss):
        assert call(filt(ss), **kw) == 1


@pytest.mark.parametrize("kw", [dict(temperature=FAKE + 2), dict(top_k=FAKE + 1), dict(top_p=FAKE + 3), dict(min_p=FAKE + 2),
                                dict(request=FAKE + 2), dict(requests=3), dict(request=FAKE, requests=0), dict(reserved=1)])
def test_bad_filters_are_refused(ss, kw):
    for call in calls(ss):
        assert call(filt(ss, **kw)) == 1
        assert call(None) == 1


def test_bad_outputs_are_refused(ss):
    mask, sample = calls(ss)
    f = filt(ss)
    assert mask(f, out=None) == 1
    assert mask(f, out=FAKE + 1) == 1
    assert mask(f, out_stride=99) == 1
    assert mask(f, out=FAKE, out_stride=104) == 1  # in place, with another stride
    assert sample(f, uniforms=None) == 1
    assert sample(f, uniforms=FAKE + 2) == 1
    assert sample(f, out_tokens=None) == 1
    assert sample(f, out_tokens=FAKE + 1) == 1
    assert sample(f, out_logprob=FAKE + 2) == 1


def test_no_rows_are_nothing_to_do(ss):
    mask, sample = calls(ss)
    f = filt(ss, requests=0)
    assert mask(f, rows=0, logits=None, out=None) == 0
    assert sample(f, rows=0, logits=None, uniforms=None, out_tokens=None) == 0


def ones(n, kind=torch.float32):
    return torch.ones(n, dtype=kind)


def test_binding_checks_filters(ss):
    with pytest.raises(TypeError):
        ss.Filter(temperature=ones(3, torch.float64))
    with pytest.raises(TypeError):
        ss.Filter(top_k=ones(3))
    with pytest.raises(ValueError):
        ss.Filter(temperature=ones(3), top_p=ones(4))
    with pytest.raises(ValueError):
        ss.Filter(temperature=ones(6)[::2])
    with pytest.raises(ValueError):
        ss.Filter(temperature=ones((3, 1)))
    with pytest.raises(ValueError):
        ss.Filter()


def test_binding_checks_tensors(ss, monkeypatch):
    class Reached(Exception):
        pass

    def stop(*args):
        raise Reached
    monkeypatch.setattr(ss.lib, "spec_filter", stop)
    monkeypatch.setattr(ss.lib, "spec_sample", stop)
    monkeypatch.setattr(ss.Filter, "_stream", lambda self, stream: None)
    f = ss.Filter(temperature=ones(4))
    i32 = torch.int32
    x = torch.zeros((4, 9))
    for good in (x, x[:2], x.bfloat16(), x[:, :5]):
        n = len(good)
        with pytest.raises(Reached):
            f.mask(good, good.clone(), ones(n, i32))
        with pytest.raises(Reached):
            f.sample(good, ones(n), ones(n, i32), ones(n), ones(n, i32))
    for bad in (x.double(), x.half(), x[0], x.T, torch.zeros((5, 9)), torch.zeros((4, 18))[:, ::2]):
        with pytest.raises((ValueError, TypeError)):
            f.mask(bad, bad.clone())
        with pytest.raises((ValueError, TypeError)):
            f.sample(bad, ones(len(bad)), ones(len(bad), i32))
    for out in (x[:3], x.bfloat16(), x[:, :8], torch.zeros((9, 4)).T):
        with pytest.raises((ValueError, TypeError)):
            f.mask(x, out)
    for kw in (dict(uniforms=ones(3)), dict(uniforms=ones(4, torch.float64)), dict(out_tokens=ones(4, torch.int64)),
               dict(out_tokens=ones(8, i32)[::2]), dict(out_logprob=ones(5)), dict(out_kept=ones(4))):
        with pytest.raises((ValueError, TypeError)):
            f.sample(x, **{**dict(uniforms=ones(4), out_tokens=ones(4, i32)), **kw})
    shared = ss.Filter(temperature=ones(2), request=torch.zeros(4, dtype=i32))
    with pytest.raises(Reached):
        shared.mask(x, x)
    with pytest.raises(ValueError):
        shared.mask(x[:3], x[:3])


def test_tensors_of_the_host_are_refused(ss):
    f, x = ss.Filter(temperature=ones(4)), torch.zeros((4, 9))
    with pytest.raises(ValueError, match="CUDA"):
        f.mask(x, x.clone())
    with pytest.raises(ValueError, match="CUDA"):
        f.sample(x, ones(4), ones(4, torch.int32))
