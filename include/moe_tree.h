/*
 * moe_tree.h -- C ABI of a verify step on a tree of drafted tokens, for AMD
 * Instinct MI355X (gfx950): the tree's plan, attention of its rows over the
 * paged 4-bit cache of moe_kv.h, and the move of the accepted path to its
 * places in the cache.  moe_sample.h verifies the tree in between.
 *
 * "Support Step3.5/3.7 flash mtp3" (Overview, data-flow trace of one MTP
 * step) verifies one chain of drafts, [id_last, draft_1, ...].  A tree keeps
 * several continuations of a token: row 0 of a sequence is the last accepted
 * token (the root), every other row a draft, and parents[i] is the row, of the
 * same sequence, that draft i follows.  A chain is the tree of parents i - 1.
 *
 * A step of a tree: moe_tree_plan once; in every layer moe_kv_append with the
 * plan's positions, then moe_kv_tree_attention with the plan's mask;
 * moe_verify_sample; moe_kv_commit for all layers' caches.  seq_lens counts
 * the tree's rows until the commit, whose kept_lens replace it.
 *
 * Status codes, ownership and ordering are those of moe_kv.h.
 */
#ifndef SVR_MOE_TREE_H
#define SVR_MOE_TREE_H

#include <stddef.h>
#include <stdint.h>

#include "moe_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_TREE_MAX_ROWS 1024    /* rows of one sequence's tree */
#define MOE_TREE_MAX_TOKENS 65536 /* rows of a call */
#define MOE_TREE_MAX_CACHES 256   /* caches of one moe_kv_commit */

/* The trees of a batch: sequence b has the rows q_offsets[b] to
 * q_offsets[b+1], those from max_rows on are no nodes.  parents[i] is the
 * place of row i's parent among its sequence's rows and has to be smaller than
 * row i's own; a row with another value hangs on nothing: it is the root of a
 * tree of its own, which is never accepted.  Row 0's is not read.  A row's
 * children are the rows that name it, in ascending order; those behind the
 * first max_children are never accepted. */
typedef struct moe_tree {
  int32_t n_seqs;       /* sequences, at most MOE_KV_MAX_SEQS */
  int32_t n_rows;       /* rows that the batch's arrays have (padding included) */
  int32_t max_rows;     /* 1 to MOE_TREE_MAX_ROWS */
  int32_t max_children; /* 1 to MOE_TREE_MAX_ROWS */
  const int32_t* q_offsets; /* [n_seqs + 1], ascending, from 0 */
  const int32_t* parents;   /* [n_rows]; NULL: chains */
} moe_tree;

/* Masks and positions of the rows, ONE launch.
 *   seq_lens  [n_seqs] tokens of each sequence with its rows, as in moe_kv.h.
 *   mask      [n_rows][mask_words] out: bit j % 64 of word j / 64 of a row is
 *             set where it sees row j of its sequence: its ancestors and itself.
 *   positions [n_rows] int32 out: seq_lens[b] - rows of b + depth of the row.
 * Either may be NULL.  Rows of no sequence, and rows from max_rows on, are left
 * as they were.  MOE_ERR_NULL: a NULL tree, q_offsets, or seq_lens with
 * positions; MOE_ERR_SHAPE: tree out of range, or mask_words * 64 < max_rows
 * with a mask, or mask_words > MOE_TREE_MAX_ROWS / 64; MOE_ERR_ARG: a pointer
 * not aligned to its elements.  n_seqs == 0 or n_rows == 0: MOE_OK. */
int32_t moe_tree_plan(const moe_tree* tree, const int32_t* seq_lens, uint64_t* mask,
                      int32_t mask_words, int32_t* positions, void* hip_stream);

/* moe_kv_attention with the new rows' places among each other given by a mask.
 * Row i of sequence b sees the tokens before its sequence's new rows, places
 * [0, base) with base = seq_lens[b] - rows of b, then the new rows (places
 * base + j, below base + max_rows) whose bit j is set in its mask, and where
 * window > 0 the last `window` tokens of this list only.  Bits need not be
 * those of a tree: bits behind the sequence's rows mean nothing, a row without
 * any sees the tokens before it, and zeros and -inf come out where it sees
 * none at all.
 *   mask [n_tokens][mask_words], 64 * mask_words >= max_rows, at most
 *   MOE_TREE_MAX_ROWS.
 * Everything else (q, out, lse, roundings, a workspace of
 * moe_kv_attention_workspace_bytes, errors) as moe_kv_attention; MOE_ERR_NULL
 * for a NULL mask, MOE_ERR_SHAPE for mask_words out of range, MOE_ERR_ARG for a
 * mask not 8-byte aligned. */
int32_t moe_kv_tree_attention(const moe_kv_desc* desc, const moe_kv_batch* batch, int32_t dtype,
                              const uint64_t* mask, int32_t mask_words, const void* q,
                              int64_t q_stride, const void* cache, int32_t n_pages, void* out,
                              float* lse, void* workspace, size_t workspace_bytes,
                              void* hip_stream);

/* The accepted path's tokens move to their places, ONE launch for all layers.
 * For each sequence b with rows, base = seq_lens[b] - rows of b, and each
 * i <= n_accepted[b]: the token at base + path[b][i] is stored at base + i, as
 * it lies.  path[b][0] is the root, 0; a path ascends, so path[b][i] >= i; an
 * entry below i or not among the sequence's rows is not moved, nor is a token
 * from or to a place that has no page.  What lies behind base + n_accepted[b] is
 * as good as free.  Pages that tokens move from or to belong to one sequence.
 *   path       [n_seqs][path_stride], path_stride >= 1 entries a sequence.
 *   n_accepted [n_seqs]; taken as path_stride - 1 or the sequence's rows - 1
 *              where it is larger, as 0 where it is negative.
 *   caches     n_caches (1 to MOE_TREE_MAX_CACHES) device pointers, in HOST
 *              memory, read before the call returns: caches of one layout, with
 *              n_pages pages each.  No two may be the same or overlap.
 *   kept_lens  [n_seqs] int32 out, may be NULL, neither seq_lens nor n_accepted:
 *              base + n_accepted[b] + 1, seq_lens[b] for a sequence without rows.
 * The trees' rows are those of the batch below max_rows.
 * MOE_ERR_NULL: a NULL struct, batch array, path, n_accepted, caches or cache.
 * MOE_ERR_SHAPE: desc, batch, n_pages, path_stride or n_caches out of range, or
 * n_seqs * n_kv_heads * n_caches 2^24 or more.  MOE_ERR_ARG: a pointer not
 * aligned to its elements, a cache not 16-byte aligned, caches that overlap, kept_lens
 * equal to seq_lens or n_accepted.  n_seqs == 0: MOE_OK. */
int32_t moe_kv_commit(const moe_kv_desc* desc, const moe_kv_batch* batch, const int32_t* path,
                      int64_t path_stride, const int32_t* n_accepted, void* const* caches,
                      int32_t n_caches, int32_t n_pages, int32_t* kept_lens, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SVR_MOE_TREE_H */
