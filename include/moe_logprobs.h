/*
 * moe_logprobs.h -- C ABI of log probabilities of given tokens, with the
 * entropy and the top alternatives of each row of logits, for AMD Instinct
 * MI355X (gfx950).  It reads the logits that moe_verify_accept
 * (moe_accept.h) reads: "Support Step3.5/3.7 flash mtp3" (Overview,
 * data-flow trace of one MTP step, steps 4 and 5) has logits on for every
 * verify row, and a server reports these numbers for the accepted tokens; a
 * prefill micro-batch gives those of the prompt.
 *
 * For each row x of V logits, with m = max x, z = sum_i e^(x_i - m):
 *   logprob[t] = x_t - m - ln z,   entropy = ln z - sum_i e^(x_i - m)(x_i - m) / z
 * (terms of weight zero count as zero).  The alternatives are the top_k
 * columns by value, equal ones by the lower column, with their logprobs; NaN
 * counts as -inf in that order and -0 as +0, as in moe_accept.h.
 *   A row that is -inf everywhere has no distribution: its logprobs are -inf
 * and its entropy 0.  A row that holds a NaN or +inf gives NaN for all of
 * them.  A target outside [0, V) is no token: its logprob is NaN.
 *
 * Status codes and ownership are those of moe_layer.h.
 */
#ifndef SVR_MOE_LOGPROBS_H
#define SVR_MOE_LOGPROBS_H

#include <stddef.h>
#include <stdint.h>

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_LOGPROBS_MAX_TOP 64
#define MOE_LOGPROBS_MAX_ROWS 1048576
#define MOE_LOGPROBS_MAX_VOCAB 1073741824 /* 2^30 columns */

/* Device workspace, in *bytes, of moe_logprobs for up to max_rows rows of
 * vocab columns and max_top alternatives: 2048 bytes of counters, then the
 * parts of rows that several workgroups share.  The counters must be zero
 * before the first call that uses the workspace; every call leaves them
 * zero, so zero-fill a workspace once when it is allocated.  Calls that
 * share a workspace must not overlap in time.
 * MOE_ERR_NULL if bytes is NULL; MOE_ERR_SHAPE for sizes out of range. */
int32_t moe_logprobs_workspace_bytes(int32_t max_rows, int64_t vocab, int32_t max_top,
                                     size_t* bytes);

/* ONE launch.  All pointers are device pointers of the caller.
 *   logits  [n_rows][vocab] of dtype (MOE_F32, MOE_BF16, MOE_F16), rows
 *           row_stride elements apart.
 *   targets [n_rows] int32, and logprobs [n_rows] float out; both or neither NULL.
 *   entropy [n_rows] float out, may be NULL.
 *   top_ids [n_rows][top_k] int32 out and top_logprobs [n_rows][top_k] float
 *           out; either may be NULL; both unused if top_k == 0.
 * Errors (nothing enqueued): MOE_ERR_NULL for NULL logits or workspace, or
 * exactly one of targets and logprobs; MOE_ERR_SHAPE for n_rows, vocab,
 * top_k > min(vocab, MOE_LOGPROBS_MAX_TOP) or row_stride < vocab;
 * MOE_ERR_DTYPE; MOE_ERR_WORKSPACE; MOE_ERR_ARG for a pointer not aligned to
 * its elements or a workspace not 256-byte aligned.  n_rows == 0: MOE_OK.
 * Sums are 32-bit, in an order that depends on the sizes alone. */
int32_t moe_logprobs(const void* logits, int32_t dtype, int32_t n_rows, int64_t vocab,
                     int64_t row_stride, const int32_t* targets, float* logprobs, float* entropy,
                     int32_t top_k, int32_t* top_ids, float* top_logprobs, void* workspace,
                     size_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SVR_MOE_LOGPROBS_H */
