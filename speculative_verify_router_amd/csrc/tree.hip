// The plan of a tree of drafts, and the move of its accepted path in the cache
// (include/moe_tree.h).  Both are bound by latency, a few loads that depend on
// each other: 3.0 us for the plan of 61 rows, 5.1 for 48 trees of up to 253 rows
// (192 workgroups, 0.2 MB); 3.0 for the path of one sequence in one cache, 7.1
// for 48 sequences in eight of eight heads (48 * 64 workgroups, 4 MB).  A call's
// host time is more, 6 us.
#include "kv.h"
#include "tree.h"

namespace svr {
namespace {

// Masks and positions by doubling: a row knows the ancestors up to its `jump`
// (exclusive), which knows as many more, so a tree of depth d takes log2 d
// rounds.  One workgroup makes one word of the masks of a sequence.
struct PlanArgs {
  TreeArgs tree;
  const int32_t* lens;
  uint64_t* mask;
  int words;
  int32_t* positions;
};

__global__ __launch_bounds__(kBlock) void k_tree_plan(PlanArgs a) {
  constexpr int kMost = MOE_TREE_MAX_ROWS;
  __shared__ uint64_t s_mask[kMost];
  __shared__ short s_jump[2][kMost], s_depth[2][kMost];
  const int b = blockIdx.x / a.words, w = blockIdx.x % a.words;
  const TreeRows s = tree_rows(a.tree, b);
  const int base = a.lens ? (int)((int64_t)a.lens[b] - s.all) : 0;
  for (int i = threadIdx.x; i < s.rows; i += blockDim.x) {
    const int p = i ? tree_parent(a.tree, s.off, i) : -1;
    s_mask[i] = i >> 6 == w ? 1ull << (i & 63) : 0;
    s_jump[0][i] = (short)p;
    s_depth[0][i] = p >= 0;
  }
  // (Uniform: every thread sees the same `more`.)
  int at = 0;
  for (bool more = true; more; at ^= 1) {
    __syncthreads();
    bool on = false;
    for (int i = threadIdx.x; i < s.rows; i += blockDim.x) {
      int j = s_jump[at][i], d = s_depth[at][i];
      if (j >= 0) {
        // The jump's mask may hold what it learns in this round already:
        // ancestors all the same.
        s_mask[i] |= s_mask[j];
        d += s_depth[at][j];
        j = s_jump[at][j];
        on |= j >= 0;
      }
      s_jump[at ^ 1][i] = (short)j;
      s_depth[at ^ 1][i] = (short)d;
    }
    more = __syncthreads_or(on);
  }
  for (int i = threadIdx.x; i < s.rows; i += blockDim.x) {
    if (a.mask) a.mask[(int64_t)(s.off + i) * a.words + w] = s_mask[i];
    if (a.positions && w == 0) a.positions[s.off + i] = base + s_depth[at][i];
  }
}

// The accepted path's tokens to their places: a workgroup moves those of one
// head in one cache.  A token's codes are pieces of 16 bytes, its scales of 2,
// a thread each; as many tokens at a time as there are threads for.  Places
// come from at or behind where they go, so what a round reads no round before
// it has written: one barrier, between a round's loads and its stores.
struct CommitArgs {
  KvArgs kv;
  const int32_t* path;
  int64_t path_stride;
  const int32_t* n_acc;
  int32_t* kept;
  int n_caches;
  uint8_t* cache[MOE_TREE_MAX_CACHES];
};

__global__ __launch_bounds__(kBlock) void k_kv_commit(CommitArgs a) {
  const int h = blockIdx.x % a.kv.Hk, x = blockIdx.x / a.kv.Hk;
  const int b = x % a.kv.n_seqs, c = x / a.kv.n_seqs;
  const int off = a.kv.offs[b], end = a.kv.offs[b + 1], len = a.kv.lens[b], wanted = a.n_acc[b];
  const int all = off >= 0 && end > off && end <= a.kv.n_tokens ? end - off : 0;
  const int rows = min(all, a.kv.max_rows);
  const int64_t base = (int64_t)len - all;
  const int n = (int)min((int64_t)max(min(wanted, rows - 1), 0), a.path_stride - 1);
  if (a.kept && h == 0 && c == 0 && threadIdx.x == 0) a.kept[b] = all ? (int32_t)(base + n + 1) : len;
  if (!rows) return;

  const int D = a.kv.D, P = 1 << a.kv.page_shift;
  const int codes = D / 32, scales = D / 64, pieces = 2 * (codes + scales);  // of a side; of a token
  const int tokens = kBlock / pieces;
  const int mine = threadIdx.x / pieces, piece = threadIdx.x - mine * pieces;
  uint8_t* cache = a.cache[c];
  // Where a piece lies, from the start of its page: of the token at place p there.
  auto at = [&](int p) {
    if (piece < 2 * codes) {
      const int side = piece >= codes, k = piece - side * codes;
      return (side * P + p) * (D / 2) + 16 * k;
    }
    const int q = piece - 2 * codes, side = q >= scales, k = q - side * scales;
    return P * D + (side * P + p) * (D / 32) + 2 * k;
  };
  const bool wide = piece < 2 * codes;
  for (int i0 = 1; i0 <= n; i0 += tokens) {
    const int i = i0 + mine;
    uint4 v = {};
    int64_t to = -1;
    if (mine < tokens && i <= n) {
      const int r = a.path[b * a.path_stride + i];
      if (r > i && r < rows) {
        const int64_t src = kv_page_base(a.kv, b, base + r, h), dst = kv_page_base(a.kv, b, base + i, h);
        if (src >= 0 && dst >= 0) {
          const uint8_t* from = cache + src + at((int)(base + r) & (P - 1));
          to = dst + at((int)(base + i) & (P - 1));
          if (wide) v = ld16(from);
          else v.x = *reinterpret_cast<const uint16_t*>(from);
        }
      }
    }
    __syncthreads();
    if (to >= 0) {
      if (wide) *reinterpret_cast<uint4*>(cache + to) = v;
      else *reinterpret_cast<uint16_t*>(cache + to) = (uint16_t)v.x;
    }
  }
}

}  // namespace
}  // namespace svr

using namespace svr;

extern "C" {

int32_t moe_tree_plan(const moe_tree* tree, const int32_t* seq_lens, uint64_t* mask,
                      int32_t mask_words, int32_t* positions, void* hip_stream) {
  const int32_t rc = tree_check(tree, true);
  if (rc != MOE_OK) return rc;
  if (mask && (mask_words < 1 || mask_words > MOE_TREE_MAX_ROWS / 64 || tree->max_rows > 64 * mask_words))
    return MOE_ERR_SHAPE;
  if (tree->n_seqs == 0 || tree->n_rows == 0) return MOE_OK;
  if (positions && !seq_lens) return MOE_ERR_NULL;
  if ((uintptr_t)mask % 8 || ((uintptr_t)positions | (uintptr_t)seq_lens) % 4) return MOE_ERR_ARG;
  if (!mask && !positions) return MOE_OK;
  PlanArgs a{tree_args(tree), seq_lens, mask, mask ? mask_words : 1, positions};
  const int threads = tree->max_rows >= kBlock ? kBlock : (tree->max_rows + kWave - 1) / kWave * kWave;
  (void)hipGetLastError();
  hipLaunchKernelGGL(k_tree_plan, dim3((unsigned)tree->n_seqs * (unsigned)a.words), dim3(threads), 0,
                     (hipStream_t)hip_stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

int32_t moe_kv_commit(const moe_kv_desc* desc, const moe_kv_batch* batch, const int32_t* path,
                      int64_t path_stride, const int32_t* n_accepted, void* const* caches,
                      int32_t n_caches, int32_t n_pages, int32_t* kept_lens, void* hip_stream) {
  int32_t rc = kv_check_desc(desc);
  if (rc == MOE_OK) rc = kv_check_batch(desc, batch, true);
  if (rc != MOE_OK) return rc;
  if (n_pages < 1 || path_stride < 1 || n_caches < 1 || n_caches > MOE_TREE_MAX_CACHES) return MOE_ERR_SHAPE;
  const int64_t grid = (int64_t)batch->n_seqs * desc->n_kv_heads * n_caches;
  if (!kv_grid_fits(grid, kBlock)) return MOE_ERR_SHAPE;
  if (batch->n_seqs == 0) return MOE_OK;
  if (!path || !n_accepted || !caches) return MOE_ERR_NULL;
  CommitArgs a{};
  const uint64_t bytes = (uint64_t)n_pages * desc->n_kv_heads * (uint64_t)kv_page_bytes(desc);
  for (int32_t c = 0; c < n_caches; ++c) {
    if (!caches[c]) return MOE_ERR_NULL;
    if ((uintptr_t)caches[c] % 16) return MOE_ERR_ARG;
    for (int32_t e = 0; e < c; ++e) {  // tokens of both would move twice, or from half written ones
      const uint64_t p = (uint64_t)(uintptr_t)caches[e], q = (uint64_t)(uintptr_t)caches[c];
      if ((p < q ? q - p : p - q) < bytes) return MOE_ERR_ARG;
    }
    a.cache[c] = (uint8_t*)caches[c];
  }
  if (((uintptr_t)path | (uintptr_t)n_accepted | (uintptr_t)kept_lens) % 4) return MOE_ERR_ARG;
  // What other workgroups still read.
  if (kept_lens && (kept_lens == batch->seq_lens || kept_lens == n_accepted)) return MOE_ERR_ARG;
  a.kv = kv_args(desc, batch, n_pages);
  a.path = path;
  a.path_stride = path_stride;
  a.n_acc = n_accepted;
  a.kept = kept_lens;
  a.n_caches = n_caches;
  (void)hipGetLastError();
  hipLaunchKernelGGL(k_kv_commit, dim3((unsigned)grid), dim3(kBlock), 0, (hipStream_t)hip_stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
