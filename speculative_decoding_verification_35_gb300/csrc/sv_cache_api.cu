// C ABI of the cache calls (include/speccache.h): host-side validation and the launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "sv_cache.cuh"

using namespace sv::cache;

namespace {

int elem_size(int dtype) { return dtype == SV_E4M3 ? 1 : 2; }

bool aligned(const void* p, size_t n) { return p && (uintptr_t)p % n == 0; }

bool valid(const sv_cache* c) {
    if (!c || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4)) return false;
    if (c->dtype != SV_BF16 && c->dtype != SV_F16 && c->dtype != SV_E4M3) return false;
    const int unit = 16 / elem_size(c->dtype);  // elements of 16 bytes
    if (c->layers < 1 || c->layers > 16384 || c->pages < 1 || c->heads < 1 || c->heads > 4096) return false;
    if (c->page_size < 8 || c->page_size > 65536 || c->page_size % 8) return false;
    if (c->head_dim < 8 || c->head_dim > 128 || c->head_dim % unit) return false;
    if (c->table_stride < 1 || c->reserved != 0) return false;
    for (int64_t s : {c->stride_page, c->stride_token, c->stride_head, c->stride_layer})
        if (s < c->head_dim || s % unit || s >= (int64_t)1 << 38) return false;
    if (c->dtype != SV_E4M3 && (c->k_scale || c->v_scale)) return false;
    return (uintptr_t)c->k_scale % 4 == 0 && (uintptr_t)c->v_scale % 4 == 0;
}

bool valid(const sv_chunk* c) {
    if (!c || c->B < 0 || c->rows < 0 || c->max_gamma < 0 || c->reserved != 0) return false;
    if (c->parents && c->max_gamma > SV_MAX_GAMMA) return false;
    if ((uintptr_t)c->parents % 4) return false;
    return c->B == 0 || (aligned(c->seq_offsets, 4) && aligned(c->cached, 4));
}

bool valid_types(int dtype, int held) { return held == SV_E4M3 ? dtype == SV_BF16 : dtype == held; }

Pool pool_of(const sv_cache* c, int32_t layer) {
    Pool p{};
    const int64_t at = (int64_t)layer * c->stride_layer * elem_size(c->dtype);
    p.k = (char*)c->k + at;
    p.v = (char*)c->v + at;
    p.k_scale = c->k_scale ? c->k_scale + (int64_t)layer * c->heads : nullptr;
    p.v_scale = c->v_scale ? c->v_scale + (int64_t)layer * c->heads : nullptr;
    p.table = c->page_table;
    p.s_page = c->stride_page;
    p.s_token = c->stride_token;
    p.s_head = c->stride_head;
    p.s_layer = c->stride_layer;
    p.pages = c->pages;
    p.page_size = c->page_size;
    p.heads = c->heads;
    p.dim = c->head_dim;
    p.table_stride = c->table_stride;
    p.layers = c->layers;
    return p;
}

// path: the accepted path of spec_cache_compact, which reads no parents.
Chunk chunk_of(const sv_chunk* c, const int32_t* path = nullptr) {
    Chunk r{};
    r.offs = c->seq_offsets;
    r.cached = c->cached;
    r.parents = c->max_gamma > 0 ? c->parents : nullptr;
    r.end = r.parents || path ? c->seq_offsets + c->B : nullptr;
    r.B = c->B;
    r.rows = c->rows;
    r.max_gamma = std::min(c->max_gamma, std::max(c->rows, 1) - 1);  // as many as there can be
    return r;
}

int result(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

}  // namespace

extern "C" {

int spec_cache_append(const sv_cache* cache, int32_t layer, const sv_chunk* chunk, const sv_rope* rope,
                      int32_t dtype, int32_t q_heads, const void* q, int64_t q_stride, const void* k, const void* v,
                      int64_t kv_stride, void* q_out, uint32_t* device_status, void* cuda_stream) {
    if (!valid(cache) || !valid(chunk) || layer < 0 || layer >= cache->layers) return SV_ERR_INVALID_ARG;
    if (!valid_types(dtype, cache->dtype)) return SV_ERR_INVALID_ARG;
    if (rope && (!aligned(rope->table, 16) || rope->positions < 1 || rope->dim < 16 || rope->dim % 16 ||
                 rope->dim > cache->head_dim || rope->reserved != 0))
        return SV_ERR_INVALID_ARG;
    if ((uintptr_t)device_status % 4) return SV_ERR_INVALID_ARG;
    const int64_t D = cache->head_dim;
    if (q && (q_heads < 1 || q_heads > 65536 || q_stride < q_heads * D || q_stride % 8)) return SV_ERR_INVALID_ARG;
    if (kv_stride < cache->heads * D || kv_stride % 8) return SV_ERR_INVALID_ARG;
    if (chunk->B == 0 || chunk->rows == 0) return SV_OK;
    if (!aligned(k, 16) || !aligned(v, 16)) return SV_ERR_INVALID_ARG;
    if (q && (!aligned(q, 16) || !aligned(q_out, 16))) return SV_ERR_INVALID_ARG;
    if (q && q == q_out && q_stride != q_heads * D) return SV_ERR_INVALID_ARG;
    AppendArgs A{};
    A.pool = pool_of(cache, layer);
    A.chunk = chunk_of(chunk);
    if (rope) {
        A.rope = rope->table;
        A.positions = rope->positions;
        A.rot = rope->dim;
    }
    A.q_heads = q ? q_heads : 0;
    A.q = q;
    A.k = k;
    A.v = v;
    A.q_stride = q_stride;
    A.kv_stride = kv_stride;
    A.q_out = q_out;
    A.status = device_status;
    return result(launch_append(A, dtype, cache->dtype, rope && rope->interleaved, (cudaStream_t)cuda_stream));
}

size_t spec_cache_workspace_size(const sv_cache* cache) {
    return valid(cache) ? attend_workspace(cache->head_dim, cache->dtype) : 0;
}

int spec_cache_attend(const sv_cache* cache, int32_t layer, const sv_chunk* chunk, int32_t dtype, int32_t q_heads,
                      const void* q, int64_t q_stride, float scale, int32_t window, void* out, float* lse,
                      uint32_t* device_status, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    return spec_cache_attend_ex(cache, layer, chunk, dtype, q_heads, q, q_stride, scale, window, out, lse, device_status,
                                workspace, workspace_bytes, nullptr, cuda_stream);
}

int spec_cache_attend_ex(const sv_cache* cache, int32_t layer, const sv_chunk* chunk, int32_t dtype, int32_t q_heads,
                         const void* q, int64_t q_stride, float scale, int32_t window, void* out, float* lse,
                         uint32_t* device_status, void* workspace, size_t workspace_bytes, const sv_debug* debug,
                         void* cuda_stream) {
    if (!valid(cache) || !valid(chunk) || layer < 0 || layer >= cache->layers) return SV_ERR_INVALID_ARG;
    if (!valid_types(dtype, cache->dtype)) return SV_ERR_INVALID_ARG;
    if (q_heads < 1 || q_heads % cache->heads || q_heads / cache->heads > 128) return SV_ERR_INVALID_ARG;
    if (q_stride < (int64_t)q_heads * cache->head_dim || q_stride % 8) return SV_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || window < 0) return SV_ERR_INVALID_ARG;
    if ((uintptr_t)lse % 4 || (uintptr_t)device_status % 4) return SV_ERR_INVALID_ARG;
    if (chunk->B == 0 || chunk->rows == 0) return SV_OK;
    if (!aligned(q, 16) || !aligned(out, 16)) return SV_ERR_INVALID_ARG;
    if (!aligned(workspace, 256) || workspace_bytes < spec_cache_workspace_size(cache)) return SV_ERR_WORKSPACE;
    AttendArgs A{};
    A.pool = pool_of(cache, layer);
    A.chunk = chunk_of(chunk);
    A.q_heads = q_heads;
    A.q = q;
    A.q_stride = q_stride;
    A.scale = scale;
    A.window = window;
    A.out = out;
    A.lse = lse;
    A.status = device_status;
    A.workspace = workspace;
    A.spin_limit = debug ? debug->spin_limit : 0;
    return result(launch_attend(A, dtype, cache->dtype, (cudaStream_t)cuda_stream));
}

int spec_cache_compact(const sv_cache* cache, const sv_chunk* chunk, const int32_t* out_num_accepted,
                       const int32_t* out_path, int32_t* out_cached, uint32_t* device_status, void* cuda_stream) {
    if (!valid(cache) || !valid(chunk)) return SV_ERR_INVALID_ARG;
    if ((uintptr_t)out_path % 4 || (uintptr_t)device_status % 4) return SV_ERR_INVALID_ARG;
    if (out_path && chunk->max_gamma > SV_MAX_GAMMA) return SV_ERR_INVALID_ARG;
    if (chunk->B == 0) return SV_OK;
    if (!aligned(out_num_accepted, 4) || !aligned(out_cached, 4)) return SV_ERR_INVALID_ARG;
    CompactArgs A{};
    A.pool = pool_of(cache, 0);
    A.chunk = chunk_of(chunk, out_path);
    A.accepted = out_num_accepted;
    A.path = out_path;
    A.now = out_cached;
    A.status = device_status;
    A.esize = elem_size(cache->dtype);
    return result(launch_compact(A, (cudaStream_t)cuda_stream));
}

}  // extern "C"
