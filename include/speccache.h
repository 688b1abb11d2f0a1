/*
 * The cache side of a verify step (part of libspecverify): the paged key/value cache that a target model
 * scores a chunk of new tokens with.
 *
 * A verify step's logits come from one pass of the target model over each sequence's chunk: the last
 * committed token and the gamma_b drafts after it ("All About Transformer Inference", the KV cache and its
 * pages, lines 25-38 and 240-245; "Accelerating Sonar through speculation", section "EAGLE" for trees).
 * Every attention layer of that pass appends the chunk's keys and values (spec_cache_append) and attends
 * (spec_cache_attend); after verification the accepted path of a token tree is moved to the front of the
 * chunk's slots (spec_cache_compact). Chunks of one token (gamma_b = 0) are plain decoding, long ones
 * prompts.
 *
 * Chunk layout: the rows of the verify step. Sequence b has T_b = seq_offsets[b+1] - seq_offsets[b] + 1
 * chunk tokens, in rows seq_offsets[b] + b .. seq_offsets[b+1] + b. Token j of it has
 *   slot      cached[b] + j                      (its place in the sequence's cache),
 *   position  cached[b] + depth(j)               (depth(j) = j in a chain; in a tree the edges to the root),
 * and cached[b] tokens lie in slots 0 .. cached[b] - 1 at positions equal to their slots. Slot s is held in
 * page page_table[b * table_stride + s / page_size] at token s % page_size.
 *
 * Every array is a DEVICE pointer owned by the caller; structures are HOST memory, read during the call. All
 * calls are asynchronous on cuda_stream, allocate nothing, synchronise nothing, and can be captured into a
 * graph. Bad arguments return SV_ERR_INVALID_ARG (or SV_ERR_WORKSPACE) before anything is launched. Findings on
 * the device set bit (1u << code) of *device_status (nullable; the caller clears it):
 *   SV_ERR_BAD_OFFSETS  seq_offsets[0] != 0, T_b outside 1 .. max_gamma + 1, rows past `rows`, parents or a path
 *                       past seq_offsets[B], a parent outside [0, j), a page id outside [0, pages), an accepted
 *                       path that is none
 *   SV_ERR_CAPACITY     cached[b] < 0, or slots cached[b] + T_b past the page table, the rotation table or 2^31 - 128; or a
 *                       batch too long for one spec_cache_attend call (2^31 pieces of 128 slots, over all kv heads;
 *                       nothing is written then)
 *   SV_ERR_TIMEOUT      a bounded wait inside the launch gave up (the outputs are then undefined)
 * A sequence with a finding fails alone: append writes nothing of it, attend writes zeros and an lse of -inf
 * (nothing where the rows themselves are bad), compact moves nothing. A bad page id fails only its tokens:
 * they are not stored, not moved, and not attended to. Where seq_offsets decreases, a row that two sequences claim
 * holds either one's result, and the other's token may be missing from its cache; SV_ERR_BAD_OFFSETS is set.
 */
#ifndef SPECCACHE_H
#define SPECCACHE_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the cache calls, beside SV_BF16 of sv_dtype. An SV_E4M3 value stands for itself times the
 * scale of its layer and head. */
enum { SV_F16 = 2, SV_E4M3 = 3 };

/*
 * The cache of a model's attention layers. Element d of head h, page p, token t, layer l lies at
 * k[l * stride_layer + p * stride_page + t * stride_token + h * stride_head + d], and v alike, so pages may be
 * [token][head][dim], [head][token][dim], or slices of a larger array. k and v 16-byte aligned, strides (in
 * elements) multiples of 16 bytes and at least head_dim. page_size: a multiple of 8 up to 65536. head_dim: a
 * multiple of 8 (16 for SV_E4M3) up to 128. Scales: float[layers][heads], SV_E4M3 only, NULL for 1.
 */
typedef struct {
    void* k;
    void* v;
    const float* k_scale;
    const float* v_scale;
    const int32_t* page_table; /* int32[B][table_stride]; entries past a sequence's last page are not read */
    int64_t stride_page;
    int64_t stride_token;
    int64_t stride_head;
    int64_t stride_layer;
    int32_t dtype; /* SV_BF16, SV_F16, SV_E4M3 */
    int32_t layers;
    int32_t pages;
    int32_t page_size;
    int32_t heads;
    int32_t head_dim;
    int32_t table_stride; /* pages a sequence may have */
    int32_t reserved;     /* 0 */
} sv_cache;

/*
 * One batch of chunks. rows: rows that the q, k, v and out arrays hold (at least seq_offsets[B] + B; the
 * offsets may be made on the device, as spec_draft_ngram does, and the arrays sized for the most there can
 * be). max_gamma: no T_b exceeds max_gamma + 1. parents: NULL for chains, else int32[seq_offsets[B]] as
 * spec_verify_tree reads it (parents[seq_offsets[b] + j - 1] of token j), and max_gamma <= SV_MAX_GAMMA.
 */
typedef struct {
    const int32_t* seq_offsets;
    const int32_t* cached;
    const int32_t* parents;
    int32_t B;
    int32_t rows;
    int32_t max_gamma;
    int32_t reserved; /* 0 */
} sv_chunk;

/*
 * Rotary positions: table float[positions][dim], row p holding cos(p f_i) for i < dim / 2 and then sin(p f_i),
 * 16-byte aligned. Elements i and dim / 2 + i of a head are a pair (interleaved == 0), or 2 i and 2 i + 1
 * (interleaved != 0); elements from dim on are not rotated. dim: a multiple of 16 up to head_dim.
 */
typedef struct {
    const float* table;
    int32_t positions;
    int32_t dim;
    int32_t interleaved;
    int32_t reserved; /* 0 */
} sv_rope;

/*
 * Rotate and append. For every chunk token: q_out = rotate(q) (q NULL: keys and values only), and the
 * token's slot of `layer` gets rotate(k) and v, in the cache's type. rope NULL: no rotation. Rotations are
 * computed in float and rounded once; SV_E4M3 stores the nearest value of x / scale, clamped to +-448 (NaN
 * stays NaN).
 * dtype (of q, k, v, q_out): the cache's, or SV_BF16 for an SV_E4M3 cache. q holds q_heads heads (any count
 * >= 1) of head_dim contiguous elements per row, rows q_stride elements apart; k and v hold cache->heads
 * heads, rows kv_stride apart (the parts of one fused projection). q_out is [rows][q_heads][head_dim],
 * and may be q itself when q_stride is q_heads * head_dim. All 16-byte aligned, strides multiples of 8.
 */
int spec_cache_append(const sv_cache* cache, int32_t layer, const sv_chunk* chunk, const sv_rope* rope,
                      int32_t dtype, int32_t q_heads, const void* q, int64_t q_stride, const void* k, const void* v,
                      int64_t kv_stride, void* q_out, uint32_t* device_status, void* cuda_stream);

/* Bytes of workspace spec_cache_attend needs on this cache (0 for an invalid one). */
size_t spec_cache_workspace_size(const sv_cache* cache);

/*
 * Attention of every chunk token, whose own keys and values are already appended, over its sequence's
 * cache: query head g reads kv head g / (q_heads / cache->heads), and
 *   out[row][g] = sum_s w_s v_s / sum_s w_s,  w_s = exp(scale * q[row][g] . k_s),  lse = log(sum_s w_s)
 * over the slots s that token j sees: all cached slots, and those chunk tokens that are j or above it (in a
 * chain: slots up to its own); with window > 0 only positions above position(j) - window. Slots that no token
 * of the chunk sees, and whatever lies in pages beyond a sequence's last token, are never read into a result,
 * NaN and infinities included. A token that sees nothing (bad pages) gets zeros and an lse of -inf.
 * Scores, the softmax's statistics and the accumulators are float. Two operands of the products are held in fewer
 * bits. The weights w_s are rounded to the precision of dtype before the product with v (for fp16 to 2^-24, with an
 * SV_E4M3 cache to 2^-17 of the row's largest where they are smaller than that allows); lse has them unrounded. With an
 * SV_E4M3 cache, q's elements under 2^-9 of their row's and head's largest are held to 2^-17 of that one. Rounding the
 * weights adds to out an error of the size of out's own rounding: relative to 64 bits 0.0018 to 0.0025 in bfloat16,
 * where rounding out alone leaves 0.0017, and 0.00022 to 0.00027 in half precision, where it leaves 0.00021.
 * q as in spec_cache_append (rotated), q_heads a multiple of cache->heads by at most 128; out is
 * [rows][q_heads][head_dim], lse (nullable) float[rows][q_heads]; rows outside every sequence are not
 * written. workspace: spec_cache_workspace_size(cache) bytes aligned to 256, not shared by calls that may
 * overlap on the GPU; its contents need no preparation.
 */
int spec_cache_attend(const sv_cache* cache, int32_t layer, const sv_chunk* chunk, int32_t dtype, int32_t q_heads,
                      const void* q, int64_t q_stride, float scale, int32_t window, void* out, float* lse,
                      uint32_t* device_status, void* workspace, size_t workspace_bytes, void* cuda_stream);

/*
 * spec_cache_attend with the verify step's debug structure (NULL: none), of which spin_limit alone is read: polls after
 * which a wait between the launch's warps gives up, 0 for the library's bound. A small value exists to exercise the
 * time-out path in tests: the launch ends once its copies and products under way have, SV_ERR_TIMEOUT is set, and the
 * outputs are undefined.
 */
int spec_cache_attend_ex(const sv_cache* cache, int32_t layer, const sv_chunk* chunk, int32_t dtype, int32_t q_heads,
                         const void* q, int64_t q_stride, float scale, int32_t window, void* out, float* lse,
                         uint32_t* device_status, void* workspace, size_t workspace_bytes, const sv_debug* debug,
                         void* cuda_stream);

/*
 * After verification, in every layer: slot cached[b] + 1 + j gets the keys and values of slot
 * cached[b] + path[j], path[j] = out_path[seq_offsets[b] + j], for j < n_b = out_num_accepted[b] (as
 * spec_verify_tree wrote them: increasing nodes in 1 .. T_b - 1), and out_cached[b] = cached[b] + n_b + 1.
 * out_path NULL: linear drafts, any number of them (a prompt kept whole: n_b = T_b - 1), nothing to move. A
 * sequence with n_b < 0 (it failed verification) keeps its cache and length. out_cached may be the chunk's own `cached` array (a second small launch then writes it).
 */
int spec_cache_compact(const sv_cache* cache, const sv_chunk* chunk, const int32_t* out_num_accepted,
                       const int32_t* out_path, int32_t* out_cached, uint32_t* device_status, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECCACHE_H */
