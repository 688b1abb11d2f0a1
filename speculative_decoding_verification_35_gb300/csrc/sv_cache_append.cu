// spec_cache_append (include/speccache.h): rotate a chunk's queries and keys by their positions and write its
// keys and values into the paged cache.
//
// A pair (x, y) at position p and frequency f becomes (x cos(pf) - y sin(pf), y cos(pf) + x sin(pf)); the
// cosines and sines come from the caller's table, one row per position, which all heads of a token share.
// Nothing is reused beyond that row, so the bound is the bytes in and out.
#include "sv_cache.cuh"

namespace sv {
namespace cache {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = to_float2<T>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    uint4 u;
    u.x = from_float2<T>(x[0], x[1]);
    u.y = from_float2<T>(x[2], x[3]);
    u.z = from_float2<T>(x[4], x[5]);
    u.w = from_float2<T>(x[6], x[7]);
    *reinterpret_cast<uint4*>(p) = u;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// The division is the definition's own (x / scale, correctly rounded), so that the stored value is the nearest.
__device__ __forceinline__ void store8_e4m3(char* p, const float (&x)[8], float scale) {
    uint2 u;
    u.x = e4m3x2(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)) |
          e4m3x2(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)) << 16;
    u.y = e4m3x2(__fdiv_rn(x[4], scale), __fdiv_rn(x[5], scale)) |
          e4m3x2(__fdiv_rn(x[6], scale), __fdiv_rn(x[7], scale)) << 16;
    *reinterpret_cast<uint2*>(p) = u;
}

// One CTA per row. A unit is 8 elements, or a pair of 8 that rotate into one another; head hh of the row is a
// query head, then a key head, then a value head.
template <typename T, bool kE4m3, bool kInter>
__global__ void __launch_bounds__(kThreads) k_cache_append(const AppendArgs A) {
    const int32_t row = blockIdx.x;
    if (row == 0 && threadIdx.x == 0) {
        const int64_t end = (int64_t)A.chunk.offs[A.chunk.B] + A.chunk.B;
        if (end > A.chunk.rows || A.chunk.offs[0] != 0) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
    }
    const int32_t b = find_seq(A.chunk, row);
    if (b < 0) return;
    int32_t cap = capacity_of(A.pool);
    if (A.rot) cap = min(cap, A.positions);
    Seq s = seq_of(A.chunk, cap, b);
    const int32_t j = row - s.row0;
    int32_t depth = j;
    if (!s.err && A.chunk.parents) {
        int32_t d;
        uint32_t above;
        bool ok;
        tree_of(A.chunk, b, s.T, d, above, ok);
        depth = __shfl_sync(0xffffffffu, d, j & 31);
        if (!ok) s.err = 1u << SV_ERR_BAD_OFFSETS;
    }
    if (s.err) {
        if (threadIdx.x == 0) report(A.status, s.err);
        return;
    }
    const int64_t place = place_of(A.pool, b, s.past + j);
    const bool store = place >= 0;
    if (!store && threadIdx.x == 0) report(A.status, 1u << SV_ERR_BAD_OFFSETS);

    const int32_t rot = A.rot, D = A.pool.dim;
    const int32_t paired = kInter ? 0 : rot >> 4;
    const int32_t units = paired + ((D - (kInter ? 0 : rot)) >> 3);
    const float* cs = A.rope + (int64_t)(s.past + depth) * rot;
    const int32_t heads = A.q_heads + 2 * A.pool.heads;
    for (int32_t i = threadIdx.x; i < heads * units; i += kThreads) {
        const int32_t hh = i / units, u = i - hh * units;
        const bool is_q = hh < A.q_heads, is_v = hh >= A.q_heads + A.pool.heads;
        const int32_t h = is_q ? hh : is_v ? hh - A.q_heads - A.pool.heads : hh - A.q_heads;
        const T* src = is_q   ? (const T*)A.q + row * A.q_stride
                       : is_v ? (const T*)A.v + row * A.kv_stride
                              : (const T*)A.k + row * A.kv_stride;
        src += (int64_t)h * D;
        const int32_t d0 = u < paired ? 8 * u : (kInter ? 8 * u : rot + 8 * (u - paired));
        const int32_t d1 = u < paired ? d0 + (rot >> 1) : -1;
        float x[8], y[8];
        load8(src + d0, x);
        if (d1 >= 0) load8(src + d1, y);
        if (!is_v) {
            if (d1 >= 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float c = __ldg(cs + d0 + e), sn = __ldg(cs + (rot >> 1) + d0 + e);
                    const float a = x[e], w = y[e];
                    x[e] = a * c - w * sn;
                    y[e] = w * c + a * sn;
                }
            } else if (kInter && d0 < rot) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float c = __ldg(cs + (d0 >> 1) + e), sn = __ldg(cs + (rot >> 1) + (d0 >> 1) + e);
                    const float a = x[2 * e], w = x[2 * e + 1];
                    x[2 * e] = a * c - w * sn;
                    x[2 * e + 1] = w * c + a * sn;
                }
            }
        }
        if (is_q) {
            T* dst = (T*)A.q_out + ((int64_t)row * A.q_heads + h) * D;
            store8(dst + d0, x);
            if (d1 >= 0) store8(dst + d1, y);
        } else if (store) {
            const int64_t at = place + h * A.pool.s_head;
            char* base = is_v ? A.pool.v : A.pool.k;
            if (kE4m3) {
                const float* scales = is_v ? A.pool.v_scale : A.pool.k_scale;
                const float sc = scales ? __ldg(scales + h) : 1.f;
                store8_e4m3(base + at + d0, x, sc);
                if (d1 >= 0) store8_e4m3(base + at + d1, y, sc);
            } else {
                store8((T*)base + at + d0, x);
                if (d1 >= 0) store8((T*)base + at + d1, y);
            }
        }
    }
}

template <typename T, bool kE4m3>
void launch(const AppendArgs& A, bool inter, cudaStream_t st) {
    if (inter) k_cache_append<T, kE4m3, true><<<A.chunk.rows, kThreads, 0, st>>>(A);
    else k_cache_append<T, kE4m3, false><<<A.chunk.rows, kThreads, 0, st>>>(A);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& A, int dtype, int cache_dtype, bool interleaved, cudaStream_t st) {
    if (cache_dtype == SV_E4M3) launch<__nv_bfloat16, true>(A, interleaved, st);
    else if (dtype == SV_F16) launch<__half, false>(A, interleaved, st);
    else launch<__nv_bfloat16, false>(A, interleaved, st);
    return cudaGetLastError();
}

}  // namespace cache
}  // namespace sv
