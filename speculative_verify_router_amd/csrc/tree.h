// Shared parts of the operators on trees of drafts (include/moe_tree.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "moe_tree.h"

namespace svr {

// What the kernels need of a batch of trees.
struct TreeArgs {
  const int32_t* offs;
  const int32_t* parents;  // NULL: chains
  int n_seqs, n_rows, max_rows, max_children;
};

// Sizes only; `arrays`: the device arrays have to be there too.
inline int32_t tree_check(const moe_tree* t, bool arrays) {
  if (!t) return MOE_ERR_NULL;
  if (t->n_seqs < 0 || t->n_seqs > MOE_KV_MAX_SEQS || t->n_rows < 0 || t->n_rows > MOE_TREE_MAX_TOKENS ||
      t->max_rows < 1 || t->max_rows > MOE_TREE_MAX_ROWS || t->max_children < 1 ||
      t->max_children > MOE_TREE_MAX_ROWS)
    return MOE_ERR_SHAPE;
  if (arrays && t->n_seqs > 0 && !t->q_offsets) return MOE_ERR_NULL;
  if (arrays && ((uintptr_t)t->q_offsets | (uintptr_t)t->parents) % 4) return MOE_ERR_ARG;
  return MOE_OK;
}

inline TreeArgs tree_args(const moe_tree* t) {
  return TreeArgs{t->q_offsets, t->parents, t->n_seqs, t->n_rows, t->max_rows, t->max_children};
}

// A sequence's rows: the first, and how many are nodes; of offsets that are
// not ascending from 0 to n_rows, none.
struct TreeRows {
  int off, rows, all;
};
__device__ __forceinline__ TreeRows tree_rows(const TreeArgs& a, int off, int end) {
  TreeRows s;
  s.off = off;
  s.all = s.off >= 0 && end > s.off && end <= a.n_rows ? end - s.off : 0;
  s.rows = min(s.all, a.max_rows);
  return s;
}
__device__ __forceinline__ TreeRows tree_rows(const TreeArgs& a, int b) {
  return tree_rows(a, a.offs[b], a.offs[b + 1]);
}

// The row that row i > 0 of a sequence follows, or -1.
__device__ __forceinline__ int tree_parent(const TreeArgs& a, int off, int i) {
  const int p = a.parents ? a.parents[off + i] : i - 1;
  return (unsigned)p < (unsigned)i ? p : -1;
}

}  // namespace svr
