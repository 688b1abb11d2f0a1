"""Rows written where they lie otherwise than the logits: nothing beside the row is read (CPU).

The kernel's own arithmetic, compiled for the host: of every alignment, size and segment the words that a whole chunk is
made of hold elements of the row alone, and all of the chunk's.
"""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdio>
#include "sv_sample_words.h"
using sv::sample::Apart;
int main() {
    long chunks = 0;
    for (int size = 2; size <= 4; size += 2) {
        const int N = 16 / size, per = 4 / size;
        for (int off = 0; off < N; ++off)
            for (int o_off = 0; o_off < N; ++o_off) {
                const Apart a{off, o_off, size, N};
                if (off == o_off) continue;  // read by whole chunks
                for (int V = 1; V <= 5 * N; ++V)
                    for (int e0 = 0; e0 < V; ++e0)
                        for (int e1 = e0 + 1; e1 <= V; ++e1) {
                            if (!(e0 == 0 || (e0 + off) % N == 0) || !(e1 == V || (e1 + off) % N == 0)) continue;  // a segment's ends
                            for (int c = a.c0(e0); c < a.c1(e1, V); ++c) {
                                const int i0 = c * N - o_off, first = a.word(c) * per - off, last = (a.word(c) + a.words()) * per - off - 1;
                                ++chunks;
                                if (i0 < e0 || i0 + N > e1) return printf("chunk %d: not the segment's\n", c), 1;
                                if (first > i0 || last < i0 + N - 1) return printf("chunk %d: elements left out\n", c), 1;
                                if (first < 0 || last >= V) {
                                    printf("size %d off %d o_off %d V %d: elements %d to %d are read\n", size, off, o_off, V, first, last);
                                    return 1;
                                }
                            }
                        }
            }
    }
    return chunks > 1000 ? 0 : 1;
}
"""


def test_nothing_beside_the_row_is_read(tmp_path):
    src, exe = tmp_path / "words.cpp", tmp_path / "words"
    src.write_text(SOURCE)
    csrc = os.path.join(ROOT, "speculative_decoding_verification_35_gb300", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(exe)])
    got = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True)
    assert got.returncode == 0, got.stdout
