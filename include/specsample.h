/*
 * Filtered distributions (part of libspecverify): temperature, top-k, top-p and min-p on rows of logits, as a draft model
 * samples its tokens from them (spec_sample), and as the verify step takes them (spec_filter).
 *
 * A verify step is exact for whatever distributions its logits stand for ("6-1편. Speculative Decoding", section 2-2: the
 * emitted tokens are distributed as the target's p, lines 859-885): filtering the target's rows and the draft's rows and
 * drawing the drafts from the filtered draft rows gives tokens of the filtered target distribution. Logits of -inf have
 * p = 0 in every verify call. The kept logits are written as they are, and a verify call divides by its own temperature: that
 * has to be the requests'. So requests that are verified in one call have one temperature, or 0, which keeps a single token
 * (any temperature of the verify call will do for those); others are verified in calls of their own.
 *
 * A row l of V logits with temperature T has weights w_i = exp((l_i - max l) / T). Its tokens are ranked by their logits,
 * the largest first, equal ones by index, those of -inf not at all. The first n of the ranking are kept:
 *   n_k  = top_k, where 1 <= top_k, else all;           S_k = sum of the first n_k weights
 *   n_p  = the least n >= 1 for which the first n weights sum to top_p S_k or more, where top_p < 1, else all
 *   n_m  = the tokens with w_i >= min(min_p, 1), where min_p > 0, else all: those with l_i >= max l + T ln(min(min_p, 1)), a
 *          sum in double
 *   n    = min(n_k, n_p, n_m)
 * T = 0 keeps the first alone. Weights are held in 64-bit fixed point (steps of 2^-44, each within 2^-31 of itself), so
 * their sums are exact and do not depend on any order: a result is the same on every call and for every batch.
 *
 * Every array is a DEVICE pointer owned by the caller; sv_filter is HOST memory, read during the call. The calls are
 * asynchronous on cuda_stream, allocate nothing, synchronise nothing, need no workspace and can be captured into a graph;
 * calls on several streams may overlap. Bad arguments return SV_ERR_INVALID_ARG before anything is launched. Findings on
 * the device set bit (1u << code) of *device_status (nullable; the caller clears it) and fail their row alone:
 *   SV_ERR_NONFINITE    a NaN or +inf logit          SV_ERR_EMPTY_ROW  all logits -inf
 *   SV_ERR_INVALID_ARG  a temperature that is negative, above 1e36, not finite, or so small that log2(e) / T is not a
 *                       float; a top_p or min_p that is NaN; a uniform outside [0, 1); a request outside [0, requests)
 */
#ifndef SPECSAMPLE_H
#define SPECSAMPLE_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The largest vocabulary of the calls below. */
#define SV_MAX_FILTER_V 262144

/*
 * What the requests of a batch ask for, an entry a request: request[row] is the entry of a row (the rows of a verify step
 * share their sequence's), or, with request NULL, the row's own number is. An array that is NULL asks for nothing
 * (temperature 1).
 */
typedef struct {
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const int32_t* request; /* int32[rows] */
    int32_t requests;       /* entries of the arrays; with request NULL at least the rows */
    int32_t reserved;       /* 0 */
} sv_filter;

/*
 * out = logits where a token is kept, -inf elsewhere; out_kept (nullable, int32[rows]) = n. A row that fails is copied as
 * it is, with n = -1. logits and out hold `rows` rows of V elements, stride and out_stride elements apart (at least V;
 * columns past V are neither read nor written), at any element alignment; where rows of both lie alike within 16 bytes
 * they are written 16 bytes at a time. out may be logits itself, with the same stride; else the two do not overlap.
 * 1 <= V <= SV_MAX_FILTER_V.
 */
int spec_filter(const void* logits, sv_dtype dtype, int32_t rows, int32_t V, int64_t stride, const sv_filter* filter,
                void* out, int64_t out_stride, int32_t* out_kept, uint32_t* device_status, void* cuda_stream);

/*
 * One token a row from its filtered distribution, by the inverse CDF in index order with the uniform u = uniforms[row] of
 * [0, 1): the first kept token i whose running weight (of the kept tokens up to i) exceeds u times the kept tokens' total.
 * out_tokens int32[rows]; out_logprob (nullable, float[rows]) = the log of its probability among the kept tokens; out_kept
 * (nullable) as in spec_filter. A row that fails gets token -1, a NaN and n = -1.
 */
int spec_sample(const void* logits, sv_dtype dtype, int32_t rows, int32_t V, int64_t stride, const sv_filter* filter,
                const float* uniforms, int32_t* out_tokens, float* out_logprob, int32_t* out_kept,
                uint32_t* device_status, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECSAMPLE_H */
