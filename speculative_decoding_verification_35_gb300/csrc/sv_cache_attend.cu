// spec_cache_attend and spec_cache_attend_scored: the launches, and the merge of items that several CTAs worked on. The
// kernels are in sv_cache_attend_wide.cuh and sv_cache_attend_few.cuh.
#include "sv_cache_attend_wide.cuh"

namespace sv {
namespace cache {

template cudaError_t launch_wide<false>(const Params&, int, int, int, cudaStream_t);

namespace {

// Items that several CTAs worked on: one warp a row, the parts in their order. Bound by the latency of a few dependent
// reads from L2, so the first parts are read along with the references, and there are warps for every row at once.
constexpr int kMergeThreads = 256;
template <typename T, int DP>
__global__ void __launch_bounds__(kMergeThreads) k_attend_merge(const __grid_constant__ Params P) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t c = blockIdx.x + 1;
    const Record rec = P.records[c];
    const int32_t i = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5);  // the item's row
    if (!rec.parts || i >= rec.tokens * P.G) return;
    const int lane = threadIdx.x & 31;
    constexpr int kPer = DP / 32, kAtOnce = 4;
    const bool in = lane * kPer < P.a.pool.dim;
    const int32_t t = i / P.G, g = i - t * P.G;
    const int32_t r = t < rec.split ? i : kTile + i - rec.split * P.G;
    // the first part is the last item of CTA c - 1, the others the first items of c, c + 1, ...
    auto slot = [&](int32_t part) { return (size_t)(part ? 2 * (c + part - 1) : 2 * (c - 1) + 1) * P.part_rows + r; };
    float x[kAtOnce][kPer];
    auto read = [&](int32_t p0) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[k][e] = 0.f;
            if (p0 + k >= rec.parts || !in) continue;
            const float* o = P.part_o + slot(p0 + k) * DP + lane * kPer;
            if (kPer == 4) *reinterpret_cast<float4*>(x[k]) = *reinterpret_cast<const float4*>(o);
            else *reinterpret_cast<float2*>(x[k]) = *reinterpret_cast<const float2*>(o);
        }
    };
    read(0);
    float2 ml = lane < rec.parts ? P.part_ml[slot(lane)] : make_float2(-INFINITY, 0.f);
    float top = ml.x;
#pragma unroll 1
    for (int32_t p = 32 + lane; p < rec.parts; p += 32) top = fmaxf(top, P.part_ml[slot(p)].x);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float l = 0.f, acc[kPer] = {}, wt = 0.f;
#pragma unroll 1
    for (int32_t p = 0; p < rec.parts; p += kAtOnce) {
        if (p % 32 == 0) {
            if (p > 0) ml = p + lane < rec.parts ? P.part_ml[slot(p + lane)] : make_float2(-INFINITY, 0.f);
            wt = p + lane >= rec.parts ? 0.f : top == -INFINITY ? 1.f : exp2_fast(ml.x - base);
            float pl = ml.y * wt;
            for (int o = 16; o; o >>= 1) pl += __shfl_xor_sync(kAll, pl, o);
            l += pl;
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const float f = __shfl_sync(kAll, wt, (p + k) & 31);
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] = p + k < rec.parts ? fmaf(f, x[k][e], acc[e]) : acc[e];
        }
        if (p + kAtOnce < rec.parts) read(p + kAtOnce);
    }
    const float vs = P.a.pool.v_scale ? P.a.pool.v_scale[rec.head] : 1.f;
    const float inv = l == 0.f ? 0.f : vs / l;
    const int64_t at = (int64_t)(rec.row0 + t) * P.a.q_heads + rec.head * P.G + g;
    if (in) {
        T* out = (T*)P.a.out + at * P.a.pool.dim + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2)
            *reinterpret_cast<uint32_t*>(out + e) = from_float2<T>(acc[e] * inv, acc[e + 1] * inv);
    }
    if (P.a.lse && lane == 0) P.a.lse[at] = l == 0.f ? -INFINITY : top * kLn2 + logf(l);
}

template <typename T>
cudaError_t merge(Params& P, cudaStream_t st, bool narrow) {
    static std::atomic<unsigned long long> allowed{~0ull};  // it asks for no shared memory
    void* args[] = {&P};
    const void* k = narrow ? (const void*)k_attend_merge<T, 64> : (const void*)k_attend_merge<T, 128>;
    const int warps = kMergeThreads / 32, rows = (int)std::min((int64_t)(P.a.chunk.max_gamma + 1) * P.G, (int64_t)P.part_rows);
    return launch_early(k, &allowed, dim3(P.ctas - 1, (rows + warps - 1) / warps), kMergeThreads, 0, st, args);
}

}  // namespace

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

// One layer's keys or values as (dim, token of the page, head, page), copied in boxes of 128 bytes by `box` tokens.
bool encode_pool(CUtensorMap* m, const Pool& p, char* base, int esize, int kind, int box) {
    const cuuint64_t dims[4] = {(cuuint64_t)p.dim, (cuuint64_t)p.page_size, (cuuint64_t)p.heads, (cuuint64_t)p.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.s_token * esize, (cuuint64_t)p.s_head * esize,
                                   (cuuint64_t)p.s_page * esize};
    const cuuint32_t boxes[4] = {(cuuint32_t)(128 / esize), (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = kind == kE4m3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : kind == kFp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encoder()(m, type, 4, base, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries as (dim, head, row), copied in boxes of 128 bytes by the heads of a group by q_box rows.
bool encode_queries(CUtensorMap* m, const AttendArgs& A, int kind, int G, int q_box) {
    const cuuint64_t dims[3] = {(cuuint64_t)A.pool.dim, (cuuint64_t)A.q_heads, (cuuint64_t)A.chunk.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)A.pool.dim * 2, (cuuint64_t)A.q_stride * 2};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)G, (cuuint32_t)q_box}, ones[3] = {1, 1, 1};
    return encoder()(m, kind == kFp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     const_cast<void*>(A.q), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_early(const void* kernel, std::atomic<unsigned long long>* allowed, dim3 grid, int threads, int smem, cudaStream_t st,
                         void** args) {
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // the devices on which the kernel may use all shared memory: setting that twice does no harm
    if (dev >= 64 || !(allowed->load() >> dev & 1u)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed->fetch_or(1ull << dev);
    }
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

namespace {
// Wide partials' row length in floats.
int part_dim(int dim, int kind) { return kind == kE4m3 || dim > 64 ? 128 : 64; }
constexpr size_t kParts = (size_t)2 * (kMaxCtas / 2) * 256;  // rows of all partials: half as many CTAs as in sv_cache_attend_few.cuh
static_assert(kParts >= (size_t)2 * kMaxCtas * kFewRows, "the other launch's partials fit");
}  // namespace

size_t attend_workspace(int dim, int cache_dtype) {
    const int dp = part_dim(dim, cache_dtype == SV_E4M3 ? kE4m3 : kBf16);
    return kParts * (dp * sizeof(float) + sizeof(float2)) + kMaxCtas * sizeof(Record);
}

cudaError_t launch_attend(const AttendArgs& A, int dtype, int cache_dtype, cudaStream_t st) {
    const int kind = cache_dtype == SV_E4M3 ? kE4m3 : dtype == SV_F16 ? kFp16 : kBf16;
    const int dp = part_dim(A.pool.dim, kind);
    Params P{};
    P.a = A;
    P.polls = A.spin_limit ? A.spin_limit : kPolls;
    P.G = A.q_heads / A.pool.heads;
    P.box = kTile;
    while (A.pool.page_size % P.box) P.box /= 2;
    P.boxes = kTile / P.box;
    P.tile_pages = kTile / A.pool.page_size;
    P.tile_rest = kTile % A.pool.page_size;
    P.wide = A.pool.dim % 16 == 0 && (uintptr_t)A.out % 32 == 0;
    char* ws = (char*)A.workspace;
    P.part_o = (float*)ws;
    P.part_ml = (float2*)(ws + kParts * dp * sizeof(float));
    P.records = (Record*)(P.part_ml + kParts);
    int dev, sms;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (!encoder()) return cudaErrorNotSupported;
    P.ctas = min(sms, kMaxCtas / 2);
    P.part_rows = 2 * kTile;
    const int n = P.ctas;
    const int64_t rows = (int64_t)(A.chunk.max_gamma + 1) * P.G;
    if (rows <= kFewRows) e = A.scored ? launch_few<true>(P, kind, (int)rows, n, st) : launch_few<false>(P, kind, (int)rows, n, st);
    else e = A.scored ? launch_wide<true>(P, kind, dp, n, st) : launch_wide<false>(P, kind, dp, n, st);
    if (e != cudaSuccess) return e;
    return kind == kFp16 ? merge<__half>(P, st, dp == 64) : merge<__nv_bfloat16>(P, st, dp == 64);
}

}  // namespace cache
}  // namespace sv
