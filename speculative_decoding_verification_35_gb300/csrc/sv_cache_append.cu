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

constexpr int kThreads = 96;

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 u, float (&x)[8]) {
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
// query head, then a key head, then a value head. A thread reads some units before it is known where they go: finding
// the row's sequence, length and page takes four dependent reads, as long as the data does. Every warp looks its row up
// for itself, so a CTA has few. Prompts of 5933 rows, 60 heads of 96, fp16: 27 us (0.77 of the copy rate) with 96
// threads, 28 with 64 or 128, 33 with 256, 41 with 256 that look up first.
template <bool kInter>
constexpr int kAhead = kInter ? 4 : 2;  // 64 bytes a thread

template <typename T, bool kE4m3, bool kInter>
__global__ void __launch_bounds__(kThreads) k_cache_append(const __grid_constant__ AppendArgs A) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t row = blockIdx.x, rot = A.rot, D = A.pool.dim;
    const int32_t paired = kInter ? 0 : rot >> 4;
    const int32_t units = paired + ((D - (kInter ? 0 : rot)) >> 3), all = (A.q_heads + 2 * A.pool.heads) * units;
    struct Unit {
        int32_t h, d0, d1;  // d1 < 0: no pair
        bool is_q, is_v;
    };
    auto unit = [&](int32_t i) {
        const int32_t hh = i / units, u = i - hh * units;
        Unit r;
        r.is_q = hh < A.q_heads;
        r.is_v = hh >= A.q_heads + A.pool.heads;
        r.h = r.is_q ? hh : r.is_v ? hh - A.q_heads - A.pool.heads : hh - A.q_heads;
        r.d0 = u < paired ? 8 * u : kInter ? 8 * u : rot + 8 * (u - paired);
        r.d1 = u < paired ? r.d0 + (rot >> 1) : -1;
        return r;
    };
    constexpr int n = kAhead<kInter>;
    uint4 x[n], y[kInter ? 1 : n];
    auto read = [&](int32_t i0) {
#pragma unroll
        for (int a = 0; a < n; ++a) {
            const int32_t i = i0 + a * kThreads;
            if (i >= all) break;
            const Unit u = unit(i);
            const T* src = u.is_q ? (const T*)A.q + row * A.q_stride : (const T*)(u.is_v ? A.v : A.k) + row * A.kv_stride;
            src += (int64_t)u.h * D;
            x[a] = *reinterpret_cast<const uint4*>(src + u.d0);
            if (!kInter && u.d1 >= 0) y[kInter ? 0 : a] = *reinterpret_cast<const uint4*>(src + u.d1);
        }
    };
    read(threadIdx.x);

    if (row == 0 && threadIdx.x == 0) {
        const int64_t end = (int64_t)A.chunk.offs[A.chunk.B] + A.chunk.B;
        if (end > A.chunk.rows || A.chunk.offs[0] != 0) report(A.status, 1u << SV_ERR_BAD_OFFSETS);
    }
    const int32_t b = find_seq(A.chunk, row);
    int32_t cap = capacity_of(A.pool);
    if (A.rot) cap = min(cap, A.positions);
    // Every sequence's offsets are looked at, also of those that no row leads to.
    if (threadIdx.x == kThreads - 1)
        for (int32_t i = row; i < A.chunk.B; i += gridDim.x) report(A.status, seq_of(A.chunk, cap, i).err);
    if (b < 0) return;
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

    const float* cs = A.rope + (int64_t)(s.past + depth) * rot;
#pragma unroll 1
    for (int32_t i0 = threadIdx.x; i0 < all; i0 += n * kThreads) {
        if (i0 != threadIdx.x) read(i0);
#pragma unroll
        for (int a = 0; a < n; ++a) {
            const int32_t i = i0 + a * kThreads;
            if (i >= all) break;
            const Unit u = unit(i);
            float p[8], q[8];
            unpack8<T>(x[a], p);
            if (!kInter && u.d1 >= 0) unpack8<T>(y[kInter ? 0 : a], q);
            if (!u.is_v) {
                if (!kInter && u.d1 >= 0) {
                    float c[8], sn[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        *reinterpret_cast<float4*>(c + e) = __ldg(reinterpret_cast<const float4*>(cs + u.d0 + e));
                        *reinterpret_cast<float4*>(sn + e) = __ldg(reinterpret_cast<const float4*>(cs + (rot >> 1) + u.d0 + e));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float v = p[e], w = q[e];
                        p[e] = v * c[e] - w * sn[e];
                        q[e] = w * c[e] + v * sn[e];
                    }
                } else if (kInter && u.d0 < rot) {
                    const float4 c = __ldg(reinterpret_cast<const float4*>(cs + (u.d0 >> 1)));
                    const float4 sn = __ldg(reinterpret_cast<const float4*>(cs + (rot >> 1) + (u.d0 >> 1)));
                    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = p[2 * e], w = p[2 * e + 1];
                        p[2 * e] = v * cc[e] - w * ss[e];
                        p[2 * e + 1] = w * cc[e] + v * ss[e];
                    }
                }
            }
            if (u.is_q) {
                T* dst = (T*)A.q_out + ((int64_t)row * A.q_heads + u.h) * D;
                store8(dst + u.d0, p);
                if (!kInter && u.d1 >= 0) store8(dst + u.d1, q);
            } else if (store) {
                const int64_t at = place + u.h * A.pool.s_head;
                char* base = u.is_v ? A.pool.v : A.pool.k;
                if (kE4m3) {
                    const float* scales = u.is_v ? A.pool.v_scale : A.pool.k_scale;
                    const float sc = scales ? __ldg(scales + u.h) : 1.f;
                    store8_e4m3(base + at + u.d0, p, sc);
                    if (!kInter && u.d1 >= 0) store8_e4m3(base + at + u.d1, q, sc);
                } else {
                    store8((T*)base + at + u.d0, p);
                    if (!kInter && u.d1 >= 0) store8((T*)base + at + u.d1, q);
                }
            }
        }
    }
}

template <typename T, bool kE4m3>
cudaError_t launch(const AppendArgs& A, bool inter, cudaStream_t st) {
    const auto kernel = inter ? k_cache_append<T, kE4m3, true> : k_cache_append<T, kE4m3, false>;
    return launch_chained(kernel, dim3(A.chunk.rows), dim3(kThreads), st, A);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& A, int dtype, int cache_dtype, bool interleaved, cudaStream_t st) {
    if (cache_dtype == SV_E4M3) return launch<__nv_bfloat16, true>(A, interleaved, st);
    return dtype == SV_F16 ? launch<__half, false>(A, interleaved, st) : launch<__nv_bfloat16, false>(A, interleaved, st);
}

}  // namespace cache
}  // namespace sv
