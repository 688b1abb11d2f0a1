// Rows that are written by the output's chunks of 16 bytes where the logits lie otherwise within 16 bytes: a chunk's elements
// come from the aligned words of 4 bytes that hold them, four, or five where the elements begin and end within a word.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define SV_WORDS_HD __host__ __device__ __forceinline__
#else
#define SV_WORDS_HD inline
#endif

namespace sv {
namespace sample {

// Elements of `size` bytes, N in 16 bytes. The row's first one is `off` elements past a boundary of 16 bytes, where words are
// numbered from, and the output's is o_off past one, where its chunks are.
struct Apart {
    int32_t off, o_off, size, N;
    // by how many bits the words' contents are shifted
    SV_WORDS_HD uint32_t shift() const { return (uint32_t)((off - o_off) * size) % 4 * 8; }
    SV_WORDS_HD int32_t words() const { return shift() ? 5 : 4; }
    // the first word of the output's chunk c
    SV_WORDS_HD int32_t word(int32_t c) const { return (c * N - o_off + off) * size / 4; }
    // The chunks c0 <= c < c1 that elements e0 to e1 - 1 of a row of V fill and whose words hold nothing but the row's.
    SV_WORDS_HD int32_t c0(int32_t e0) const { return ((shift() && e0 < 1 ? 1 : e0) + o_off + N - 1) / N; }
    SV_WORDS_HD int32_t c1(int32_t e1, int32_t V) const { return ((shift() && e1 > V - 1 ? V - 1 : e1) + o_off) / N; }
};

}  // namespace sample
}  // namespace sv
