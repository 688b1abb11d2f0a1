"""speccache.h as a C and a C++ program uses it (CPU)."""
import os
import subprocess

import pytest

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
CALLER = """
#include "speccache.h"
int step(const sv_cache* c, const sv_chunk* t, const sv_rope* r, void* q, void* k, void* v, void* out, float* lse,
         int32_t* n, uint32_t* status, void* ws, size_t bytes, void* stream) {
    int rc = spec_cache_append(c, 0, t, r, SV_F16, 32, q, 4096, k, v, 1024, q, status, stream);
    rc |= spec_cache_append(c, 0, t, r, SV_BF16, 32, q, 4096, k, v, 1024, q, status, stream);
    rc |= spec_cache_attend(c, 0, t, SV_F16, 32, q, 4096, 0.1f, 0, out, lse, status, ws, bytes, stream);
    rc |= spec_cache_attend(c, 0, t, SV_BF16, 32, q, 4096, 0.1f, 0, out, lse, status, ws, bytes, stream);
    return rc | spec_cache_compact(c, t, n, n, n, status, stream);
}
"""


@pytest.mark.parametrize("compiler,suffix", [(["gcc", "-std=c99"], "c"), (["g++", "-std=c++17"], "cpp")])
def test_a_caller_names_the_types_as_they_are(tmp_path, compiler, suffix):
    src = tmp_path / f"caller.{suffix}"
    src.write_text(CALLER)
    subprocess.check_call(compiler + ["-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", INCLUDE, str(src)])
