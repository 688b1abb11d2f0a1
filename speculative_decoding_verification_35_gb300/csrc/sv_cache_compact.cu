// spec_cache_compact (include/speccache.h): after a token tree's verification, move the accepted path's keys
// and values to the front of the chunk's slots, in every layer.
//
// A path's nodes increase, so node path[j] > j + 1 or path[j] == j + 1 (nothing to move), and the slot written
// for j is never read for a later one: path[i] >= i + 1 > j + 1 for i > j. One thread therefore owns 16 bytes
// of a token (a column) and moves that column of all path tokens in order, reading a few ahead: no two threads
// touch the same bytes, and no barrier is needed. Bound by the bytes moved, and for small batches by three
// dependent loads (the count and path, the page ids, the data). 64 trees of 1 to 32 nodes, 24 layers, 8 heads of 128
// (16 MB read and written): 6.2 us, a launch's own time is 5.5.
#include "sv_cache.cuh"

namespace sv {
namespace cache {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;

// grid: (B, layers * 2, columns of a token / kThreads)
__global__ void __launch_bounds__(kThreads) k_cache_compact(const __grid_constant__ CompactArgs A, bool write_now) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int32_t b = blockIdx.x, layer = blockIdx.y >> 1;
    const Seq s = seq_of(A.chunk, capacity_of(A.pool), b);
    const int32_t n = A.accepted[b];
    uint32_t err = s.err;
    bool moves = false;
    int32_t node = 0;
    if (!err && n >= 0) {
        if (n >= s.T || (A.path && n > SV_MAX_GAMMA)) err = 1u << SV_ERR_BAD_OFFSETS;
        else if (A.path) {
            if (lane < n) node = A.path[s.row0 - b + lane];
            const int32_t before = __shfl_up_sync(0xffffffffu, node, 1);
            const bool good = lane >= n || (node > (lane ? before : 0) && node < s.T);
            if (!__all_sync(0xffffffffu, good)) err = 1u << SV_ERR_BAD_OFFSETS;
            else moves = true;
        }
    }
    const bool first = blockIdx.z == 0 && blockIdx.y == 0 && threadIdx.x == 0;
    if (first) {
        report(A.status, err);
        if (write_now) A.now[b] = err || n < 0 ? A.chunk.cached[b] : s.past + n + 1;
    }
    if (!moves) return;

    int64_t from = -1, to = -1;
    if (lane < n && node != lane + 1) {
        from = place_of(A.pool, b, s.past + node);
        to = place_of(A.pool, b, s.past + lane + 1);
        if (from < 0 || to < 0) {
            from = to = -1;
            if (blockIdx.z == 0 && blockIdx.y == 0 && threadIdx.x < 32) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
        }
    }
    const unsigned todo = __ballot_sync(0xffffffffu, from >= 0);
    const int32_t per_head = A.pool.dim * A.esize / 16;
    const int32_t col = blockIdx.z * kThreads + threadIdx.x;
    const bool mine = col < A.pool.heads * per_head;
    const int32_t h = col / per_head;
    const int64_t off = (layer * A.pool.s_layer + h * A.pool.s_head) * A.esize + (int64_t)(col - h * per_head) * 16;
    char* base = (blockIdx.y & 1 ? A.pool.v : A.pool.k) + off;
    for (unsigned left = todo; left;) {  // every lane of the warp has the same `left`
        uint4 x[kAhead];
        unsigned w = left;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (w) {
                const int64_t at = __shfl_sync(0xffffffffu, from, __ffs(w) - 1);
                if (mine) x[i] = *reinterpret_cast<const uint4*>(base + at * A.esize);
                w &= w - 1;
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (left) {
                const int64_t at = __shfl_sync(0xffffffffu, to, __ffs(left) - 1);
                if (mine) *reinterpret_cast<uint4*>(base + at * A.esize) = x[i];
                left &= left - 1;
            }
        }
    }
}

// The new lengths, written after the moves where they replace the lengths that the moves read.
__global__ void __launch_bounds__(kThreads) k_cache_advance(const __grid_constant__ CompactArgs A) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t warp = (blockIdx.x * kThreads + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (warp >= A.chunk.B) return;
    const Seq s = seq_of(A.chunk, capacity_of(A.pool), warp);
    const int32_t n = A.accepted[warp];
    bool good = !s.err && n >= 0 && n < s.T && (!A.path || n <= SV_MAX_GAMMA);
    if (good && A.path) {
        const int32_t node = lane < n ? A.path[s.row0 - warp + lane] : 0;
        const int32_t before = __shfl_up_sync(0xffffffffu, node, 1);
        good = __all_sync(0xffffffffu, lane >= n || (node > (lane ? before : 0) && node < s.T));
    }
    if (lane == 0 && good) A.now[warp] = s.past + n + 1;
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& A, cudaStream_t st) {
    const bool in_place = A.now == A.chunk.cached;
    const int32_t cols = A.pool.heads * (A.pool.dim * A.esize / 16);
    const dim3 grid((unsigned)A.chunk.B, A.path ? 2u * (unsigned)A.pool.layers : 1u,
                    A.path ? (unsigned)((cols + kThreads - 1) / kThreads) : 1u);
    const cudaError_t e = launch_chained(k_cache_compact, grid, dim3(kThreads), st, A, !in_place);
    if (e != cudaSuccess || !in_place) return e;
    return launch_chained(k_cache_advance, dim3((A.chunk.B + kThreads / 32 - 1) / (kThreads / 32)), dim3(kThreads), st, A);
}

}  // namespace cache
}  // namespace sv
