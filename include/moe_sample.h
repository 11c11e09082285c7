/*
 * moe_sample.h -- C ABI of sampled verification for AMD Instinct MI355X
 * (gfx950): drafts are accepted so that what a sequence receives is
 * distributed as the target's own tokens are.  It reads the logits that
 * moe_verify_accept (moe_accept.h) reads, of chains or trees of drafts
 * (moe_tree.h), of one or many sequences; all random numbers are inputs.
 *
 * The target's distribution after row n of a sequence with temperature T:
 *   p(x) = e^(l_x / T) / sum_y e^(l_y / T).
 * NaN, -inf and the lowest float have probability zero, +inf counts as the
 * largest float.  A temperature above 2^64 counts as that; one below 2^-126 (0,
 * negative) or NaN is greedy: p is one for the largest logit (the lowest column
 * of equal ones) and zero elsewhere, and no random number matters.
 *
 * From the root on, a row's children (moe_tree.h) are tried in ascending
 * order.  Child k has the token x_k and the random number u_k in [0, 1).
 *   Given drafts (draft_probs NULL; the draft model's best tokens, whatever
 * they were chosen by): with S = 1 at first, x_k is accepted if
 * u_k S < p(x_k), else S becomes S - p(x_k) and p(x_k) zero.
 *   Drawn drafts (x_k drawn from q, the row's draft probabilities, each
 * anew): x_k is accepted if u_k q(x_k) S < w(x_k), with w = p, S = 1 at first;
 * else w becomes (p - c q)+ and S the sum of that, with c = 1 after the first
 * rejection and c + S after the next (w / S is then the normalised positive
 * part of what it was less q).  NaN and negative q count as zero.
 * A draft whose token is outside [0, vocab) is not accepted and changes nothing.
 *   The first accepted child is the next row; the row where none is accepted
 * (or that has none) gives one more token: the first column whose cumulative
 * weight is above sample_u[b] times the sum of what is left of p, or of w.
 * Where nothing is left it is the target's most likely token; -1 where the row
 * has no distribution (no logit that counts), after which nothing is accepted.
 *
 * Weights (to 1e-13 of them), sums and comparisons are 64-bit, in an order that
 * depends on the sizes alone: borders of the cumulative sum lie closer than 32
 * bits resolve.
 * Status codes, ownership and ordering are those of moe_layer.h.
 */
#ifndef SVR_MOE_SAMPLE_H
#define SVR_MOE_SAMPLE_H

#include <stddef.h>
#include <stdint.h>

#include "moe_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_SAMPLE_MAX_ROWS 16384       /* rows and sequences of a call */
#define MOE_SAMPLE_MAX_VOCAB 1073741824 /* 2^30 columns */

/* Device workspace, in *bytes, of moe_verify_sample for trees of up to these
 * n_seqs and n_rows (the arrays may be NULL) and up to vocab columns.  It begins
 * with 131072 bytes of counters, which must be zero before the first call that
 * uses the workspace; every call leaves them zero, so zero-fill a workspace
 * once when it is allocated.  Calls that share one must not overlap in time.
 * MOE_ERR_NULL, MOE_ERR_SHAPE as below. */
int32_t moe_sample_workspace_bytes(const moe_tree* tree, int64_t vocab, size_t* bytes);

/* One launch for given drafts, 1 + max_children for drawn ones.
 *   logits      [n_rows][vocab] of dtype (MOE_F32, MOE_BF16, MOE_F16), rows
 *               row_stride elements apart: the target's logits after each row.
 *   tokens      [n_rows] int32: the rows' own tokens (those of roots not read).
 *   draft_probs [n_rows][vocab] float, rows draft_stride elements apart, or
 *               NULL: row n is what the children of row n were drawn from; rows
 *               without children are not read.
 *   temperature [n_seqs] float, NULL: 1.
 *   accept_u    [n_rows] float in [0, 1): u of each draft (roots' not read).
 *   sample_u    [n_seqs] float in [0, 1).
 *   verify_h    [n_rows][h_dim] float, may be NULL (then h_dim must be 0): the
 *               target's hidden state of each row.
 *   accepted    [n_seqs][max_rows] int32 out: the accepted drafts' tokens, the
 *               one more token, then -1.
 *   path        [n_seqs][max_rows] int32 out, may be NULL: the accepted rows
 *               (places among the sequence's rows) from the root, 0, on, then -1.
 *   n_accepted  [n_seqs] int32 out: accepted drafts.
 *   pending_h   [n_seqs][h_dim] float out: verify_h of the last row of the path.
 * Outputs of a sequence without rows are left as they were, and must not alias
 * inputs or each other.
 * Errors (nothing enqueued): MOE_ERR_NULL for a NULL tree, q_offsets, logits,
 * tokens, accept_u, sample_u, accepted, n_accepted or workspace, or exactly one
 * of verify_h and pending_h; MOE_ERR_SHAPE for tree, vocab, h_dim < 0 (or > 0
 * without verify_h), row_stride or draft_stride < vocab out of range, or more
 * than MOE_SAMPLE_MAX_ROWS rows or sequences; MOE_ERR_DTYPE; MOE_ERR_WORKSPACE;
 * MOE_ERR_ARG for a pointer not aligned to its elements or a workspace not
 * 256-byte aligned.  n_rows == 0 or n_seqs == 0: MOE_OK. */
int32_t moe_verify_sample(const moe_tree* tree, const void* logits, int32_t dtype, int64_t vocab,
                          int64_t row_stride, const int32_t* tokens, const float* draft_probs,
                          int64_t draft_stride, const float* temperature, const float* accept_u,
                          const float* sample_u, const float* verify_h, int32_t h_dim,
                          int32_t* accepted, int32_t* path, int32_t* n_accepted, float* pending_h,
                          void* workspace, size_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SVR_MOE_SAMPLE_H */
