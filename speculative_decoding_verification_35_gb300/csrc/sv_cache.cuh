// Shared by the cache kernels (include/speccache.h): their parameters, the chunk layout on the device, and
// conversions.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/speccache.h"

namespace sv {
namespace cache {

// One layer of the cache, strides in elements.
struct Pool {
    char* k;
    char* v;
    const float* k_scale;  // of the layer, [heads], or nullptr
    const float* v_scale;
    const int32_t* table;
    int64_t s_page, s_token, s_head, s_layer;
    int32_t pages, page_size, heads, dim, table_stride, layers;
};

struct Chunk {
    const int32_t* offs;
    const int32_t* cached;
    const int32_t* parents;
    const int32_t* end;  // the last offset, where an array of that many entries (parents, paths) is read; else nullptr
    int32_t B, rows, max_gamma;
};

struct AppendArgs {
    Pool pool;
    Chunk chunk;
    const float* rope;
    int32_t positions, rot;
    int32_t q_heads;  // 0: no queries
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride, kv_stride;
    void* q_out;
    uint32_t* status;
};

struct AttendArgs {
    Pool pool;
    Chunk chunk;
    int32_t q_heads;
    const void* q;
    int64_t q_stride;
    float scale;
    int32_t window;
    void* out;
    float* lse;
    uint32_t* status;
    void* workspace;
    uint32_t spin_limit;  // polls of a wait, 0: the kernels' own bound
    bool scored;          // one of these is given
    float cap;            // 0: none
    const float* slopes;  // [q_heads] or nullptr
    const int32_t* prefix;  // [B] or nullptr
};

struct CompactArgs {
    Pool pool;  // layer 0
    Chunk chunk;
    const int32_t* accepted;
    const int32_t* path;
    int32_t* now;
    uint32_t* status;
    int32_t esize;
};

struct ReserveArgs {
    int32_t* table;
    int32_t* queue;
    const int32_t* held;
    const int32_t* state;
    int32_t* out_held;
    int32_t* out_state;
    int32_t table_stride, page_size, pages;
    Chunk chunk;             // where there are no lengths
    const int32_t* lengths;
    int32_t B;
    int64_t* slots;
    uint32_t* status;
    uint32_t page_recip;  // set by the launch: a division by page_size is a product and a shift
    int32_t page_bits;
};
constexpr int32_t kMaxReserve = 1 << 16;  // sequences of a call

size_t attend_workspace(int dim, int cache_dtype);  // bytes
cudaError_t launch_append(const AppendArgs& A, int dtype, int cache_dtype, bool interleaved, cudaStream_t st);
cudaError_t launch_attend(const AttendArgs& A, int dtype, int cache_dtype, cudaStream_t st);
cudaError_t launch_compact(const CompactArgs& A, cudaStream_t st);
cudaError_t launch_reserve(const ReserveArgs& A, cudaStream_t st);

// One sequence's chunk. err: bits of the sequence's findings; rows_ok: its rows can be written.
struct Seq {
    int32_t row0, T, past;
    uint32_t err;
    bool rows_ok;
};

__device__ __forceinline__ Seq seq_of(const Chunk& c, int32_t capacity, int32_t b) {
    Seq s;
    const int64_t o0 = c.offs[b], o1 = c.offs[b + 1];
    const int32_t end = c.end ? *c.end : 0x7fffffff;
    s.past = c.cached[b];
    s.row0 = (int32_t)(o0 + b);
    s.T = (int32_t)(o1 - o0 + 1);
    s.err = 0;
    s.rows_ok = o0 >= 0 && o1 >= o0 && o1 - o0 <= c.max_gamma && o1 + b + 1 <= c.rows && o1 <= end &&
                (b > 0 || o0 == 0);
    if (!s.rows_ok) s.err = 1u << SV_ERR_BAD_OFFSETS;
    else if (s.past < 0 || (int64_t)s.past + s.T > capacity) s.err = 1u << SV_ERR_CAPACITY;
    return s;
}

// Slots a sequence may have. At most 2^31 - 128, so that the end of a tile of 128 slots is an int32 too: a table may name
// a page many times, and so be that long on any pool.
__device__ __forceinline__ int32_t capacity_of(const Pool& p) {
    const int64_t n = (int64_t)p.table_stride * p.page_size;
    return n > 0x7fffff80 ? 0x7fffff80 : (int32_t)n;
}

// The sequence of a row, by a whole warp: the last b with offs[b] + b <= row, 32 candidates a step. -1: the
// row lies in none. With inconsistent offsets it is some sequence, whose own check (seq_of) then decides.
__device__ __forceinline__ int32_t find_seq(const Chunk& c, int32_t row) {
    const int lane = threadIdx.x & 31;
    int32_t lo = 0, n = c.B;  // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int32_t step = (n + 31) >> 5;
        const int32_t b = lo + lane * step;
        const bool ok = b < lo + n && (int64_t)c.offs[b] + b <= row;
        const unsigned m = __ballot_sync(0xffffffffu, ok);
        if (!m) return -1;
        const int top = 31 - __clz(m);
        const int32_t next = lo + top * step;
        n = min(step, lo + n - next);
        lo = next;
    }
    return (int64_t)c.offs[lo] + lo <= row && row <= (int64_t)c.offs[lo + 1] + lo ? lo : -1;
}

// A tree of T <= 32 nodes, by a whole warp: lane j's depth and ancestors-or-self (bit i: node i), by
// doubling the jump to an ancestor five times. ok: every parent lies in [0, j).
__device__ __forceinline__ void tree_of(const Chunk& c, int32_t b, int32_t T, int32_t& depth, uint32_t& above,
                                        bool& ok) {
    const int lane = threadIdx.x & 31;
    int32_t p = 0;
    if (lane > 0 && lane < T) p = c.parents[(int64_t)c.offs[b] + lane - 1];
    ok = __all_sync(0xffffffffu, lane == 0 || lane >= T || (p >= 0 && p < lane));
    if (!ok) p = 0;
    depth = lane > 0 && lane < T;
    above = 1u << lane;
    if (lane > 0) above |= 1u << p;
#pragma unroll
    for (int r = 0; r < 5; ++r) {
        depth += __shfl_sync(0xffffffffu, depth, p);
        above |= __shfl_sync(0xffffffffu, above, p);
        p = __shfl_sync(0xffffffffu, p, p);
    }
}

// Byte-free address arithmetic of a token: elements from the layer's base, or -1 for a bad page id.
__device__ __forceinline__ int64_t place_of(const Pool& p, int32_t b, int32_t slot) {
    const int32_t i = slot / p.page_size;
    const int32_t id = p.table[(int64_t)b * p.table_stride + i];
    if (id < 0 || id >= p.pages) return -1;
    return id * p.s_page + (int64_t)(slot - i * p.page_size) * p.s_token;
}

__device__ __forceinline__ void report(uint32_t* status, uint32_t bits) {
    if (status && bits) atomicOr(status, bits);
}

template <typename T>
__device__ __forceinline__ float2 to_float2(uint32_t u);
template <>
__device__ __forceinline__ float2 to_float2<__nv_bfloat16>(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 to_float2<__half>(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <typename T>
__device__ __forceinline__ uint32_t from_float2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t from_float2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t from_float2<__half>(float lo, float hi) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// A launch whose CTAs may be brought in while the kernel before it in the stream ends: they wait for its end, and
// its writes, with griddepcontrol.wait before they read anything.
template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t st, Args... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace cache
}  // namespace sv
