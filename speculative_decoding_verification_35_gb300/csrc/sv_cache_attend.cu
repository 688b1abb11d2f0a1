// spec_cache_attend (include/speccache.h): attention of a chunk of new tokens over the paged cache.
//
// One pass over a row's visible slots with the running maximum m and sum l of the softmax: a batch of scores
// s_i raises m to m', and what was summed so far is scaled by exp(m - m').
#include "sv_cache.cuh"

namespace sv {
namespace cache {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDim = 128;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ float to_float(T x) {
    return (float)x;
}

// One warp per (row, query head).
template <typename T, typename C>
__global__ void __launch_bounds__(kThreads) k_attend_simple(const AttendArgs A) {
    __shared__ float qs[kWarps][kMaxDim];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int32_t row = blockIdx.x, g = blockIdx.y * kWarps + w;
    if (g >= A.q_heads) return;
    const bool one = g == 0 && lane == 0;
    if (row == 0 && one) {
        const int64_t end = (int64_t)A.chunk.offs[A.chunk.B] + A.chunk.B;
        if (end > A.chunk.rows || A.chunk.offs[0] != 0) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
    }
    const int32_t b = find_seq(A.chunk, row);
    if (b < 0) return;
    Seq s = seq_of(A.chunk, capacity_of(A.pool), b);
    const int32_t j = row - s.row0, D = A.pool.dim;
    int32_t depth_j = j, my_depth = 0;
    uint32_t above = 0;
    const bool tree = A.chunk.parents != nullptr;
    if (!s.err && tree) {
        bool ok;
        uint32_t mine;
        tree_of(A.chunk, b, s.T, my_depth, mine, ok);
        depth_j = __shfl_sync(0xffffffffu, my_depth, j & 31);
        above = __shfl_sync(0xffffffffu, mine, j & 31);
        if (!ok) s.err = 1u << SV_ERR_BAD_OFFSETS;
    }
    if (one) report(A.status, s.err);
    if (!s.rows_ok) return;
    const int32_t h = g / (A.q_heads / A.pool.heads);
    const T* q = (const T*)A.q + row * A.q_stride + (int64_t)g * D;
    for (int d = lane; d < kMaxDim; d += 32) qs[w][d] = d < D ? to_float(q[d]) : 0.f;
    __syncwarp();
    float m = -INFINITY, l = 0.f, acc[kMaxDim / 32] = {};
    const float ks = A.pool.k_scale ? A.pool.k_scale[h] : 1.f, vs = A.pool.v_scale ? A.pool.v_scale[h] : 1.f;
    const int32_t end = s.err ? 0 : s.past + j + 1;
    const int32_t pos = s.past + depth_j;
    const int32_t low = A.window > 0 ? max(0, pos - A.window + 1) : 0;
    for (int32_t k0 = low & ~31; k0 < end; k0 += 32) {
        const int32_t slot = k0 + lane, i = slot - s.past;
        const int32_t dep = __shfl_sync(0xffffffffu, my_depth, i & 31);
        bool seen = slot < end && (i < 0 ? slot >= low : (!tree || (above >> i & 1)));
        if (seen && i >= 0 && A.window > 0) seen = depth_j - (tree ? dep : i) < A.window;
        int64_t at = -1;
        if (seen) {
            at = place_of(A.pool, b, slot);
            if (at < 0) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
        }
        float x = -INFINITY;
        if (at >= 0) {
            const C* k = (const C*)A.pool.k + at + h * A.pool.s_head;
            float dot = 0.f;
            for (int d = 0; d < D; ++d) dot = fmaf(qs[w][d], to_float(k[d]), dot);
            x = dot * ks * A.scale;
        }
        float top = x;  // a NaN score stays out of the maximum and makes the sum NaN
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(m, top);
        const float base = top == -INFINITY ? 0.f : top;
        const float e = at >= 0 ? exp2f((x - base) * kLog2e) : 0.f;
        const float r = exp2f((m - base) * kLog2e);
        float sum = e;
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * r + sum;
        m = top;
#pragma unroll
        for (int c = 0; c < kMaxDim / 32; ++c) acc[c] *= r;
        for (int t = 0; t < 32; ++t) {
            const int64_t from = __shfl_sync(0xffffffffu, at, t);
            const float p = __shfl_sync(0xffffffffu, e, t);
            if (from < 0) continue;
            const C* v = (const C*)A.pool.v + from + h * A.pool.s_head;
#pragma unroll
            for (int c = 0; c < kMaxDim / 32; ++c)
                if (c * 32 + lane < D) acc[c] = fmaf(p, to_float(v[c * 32 + lane]), acc[c]);
        }
    }
    T* out = (T*)A.out + ((int64_t)row * A.q_heads + g) * D;
#pragma unroll
    for (int c = 0; c < kMaxDim / 32; ++c)
        if (c * 32 + lane < D) out[c * 32 + lane] = (T)(l == 0.f ? 0.f : acc[c] * vs / l);
    if (A.lse && lane == 0) A.lse[(int64_t)row * A.q_heads + g] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_attend(const AttendArgs& A, int dtype, int cache_dtype, cudaStream_t st) {
    const dim3 grid((unsigned)A.chunk.rows, (unsigned)((A.q_heads + kWarps - 1) / kWarps));
    if (cache_dtype == SV_E4M3) k_attend_simple<__nv_bfloat16, __nv_fp8_e4m3><<<grid, kThreads, 0, st>>>(A);
    else if (dtype == SV_F16) k_attend_simple<__half, __half><<<grid, kThreads, 0, st>>>(A);
    else k_attend_simple<__nv_bfloat16, __nv_bfloat16><<<grid, kThreads, 0, st>>>(A);
    return cudaGetLastError();
}

}  // namespace cache
}  // namespace sv
