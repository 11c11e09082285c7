// Shared parts of the paged 4-bit key/value cache (include/moe_kv.h): argument
// checks on the host, cache addresses and element types on the device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "moe_kv.h"

namespace svr {

typedef __bf16 bf16;
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));

// What the kernels need of desc and batch.
struct KvArgs {
  const int32_t* offs;
  const int32_t* lens;
  const int32_t* table;
  int n_seqs, n_tokens, max_rows, pages_per_seq;
  int Hq, Hk, D, page_shift, window, n_pages;
  int64_t page_bytes;  // of one key/value head
};

inline int kv_elem_size(int32_t dtype) {
  return dtype == MOE_F32 ? 4 : dtype == MOE_BF16 || dtype == MOE_F16 ? 2 : 0;
}

inline int32_t kv_check_desc(const moe_kv_desc* d) {
  if (!d) return MOE_ERR_NULL;
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 192 && d->head_dim != 256)
    return MOE_ERR_SHAPE;
  if (d->n_kv_heads < 1 || d->n_heads < 1 || d->n_heads > MOE_KV_MAX_HEADS ||
      d->n_heads % d->n_kv_heads)
    return MOE_ERR_SHAPE;
  if (d->page_size < 16 || d->page_size > 1024 || (d->page_size & (d->page_size - 1)))
    return MOE_ERR_SHAPE;
  if (d->window < 0 || d->rotary_dims < 0 || d->rotary_dims > d->head_dim || d->rotary_dims % 16)
    return MOE_ERR_SHAPE;
  if (d->flags & ~MOE_KV_ROTARY_INTERLEAVED) return MOE_ERR_ARG;
  if (!(d->scale >= 0.f) || !(d->norm_eps >= 0.f) || d->scale > 3e38f || d->norm_eps > 3e38f)
    return MOE_ERR_ARG;
  return MOE_OK;
}

// Sizes only; `arrays`: the device arrays have to be there too.
inline int32_t kv_check_batch(const moe_kv_desc* d, const moe_kv_batch* b, bool arrays) {
  if (!b) return MOE_ERR_NULL;
  if (b->n_seqs < 0 || b->n_seqs > MOE_KV_MAX_SEQS || b->n_tokens < 0 ||
      b->n_tokens > MOE_KV_MAX_TOKENS || b->max_rows < 0 || b->max_rows > MOE_KV_MAX_TOKENS ||
      b->pages_per_seq < 1 || (int64_t)b->pages_per_seq * d->page_size > MOE_KV_MAX_TOKENS)
    return MOE_ERR_SHAPE;
  if (arrays && b->n_seqs > 0 && (!b->q_offsets || !b->seq_lens || !b->page_table))
    return MOE_ERR_NULL;
  if (arrays && (((uintptr_t)b->q_offsets | (uintptr_t)b->seq_lens | (uintptr_t)b->page_table) % 4))
    return MOE_ERR_ARG;
  return MOE_OK;
}

// A launch has fewer than 2^32 threads.
inline bool kv_grid_fits(int64_t workgroups, int threads) { return workgroups < ((int64_t)1 << 32) / threads; }

inline int64_t kv_page_bytes(const moe_kv_desc* d) {
  return (int64_t)d->page_size * (d->head_dim + d->head_dim / 16);
}

inline KvArgs kv_args(const moe_kv_desc* d, const moe_kv_batch* b, int32_t n_pages) {
  KvArgs a{};
  a.offs = b->q_offsets;
  a.lens = b->seq_lens;
  a.table = b->page_table;
  a.n_seqs = b->n_seqs;
  a.n_tokens = b->n_tokens;
  a.max_rows = b->max_rows;
  a.pages_per_seq = b->pages_per_seq;
  a.Hq = d->n_heads;
  a.Hk = d->n_kv_heads;
  a.D = d->head_dim;
  a.page_shift = __builtin_ctz((unsigned)d->page_size);
  a.window = d->window < 1 << 30 ? d->window : 1 << 30;  // places are below 2^28: no sum passes 32 bits
  a.n_pages = n_pages;
  a.page_bytes = kv_page_bytes(d);
  return a;
}

// The sequence of row i (the last with offs[b] <= i, so never an empty one),
// or -1 for a row of no sequence.  A wave probes 64 offsets at a time.
__device__ __forceinline__ int kv_sequence_of(const KvArgs& a, int i) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, n = a.n_seqs + 1;
  while (n > 1) {
    const int step = (n + kWave - 1) / kWave;
    const int at = lane * step;
    const bool below = at < n && a.offs[lo + at] <= i;
    const int cnt = __popcll(__ballot(below));
    if (cnt == 0) return -1;
    lo += (cnt - 1) * step;
    n = min(step, n - (cnt - 1) * step);
  }
  if (a.offs[lo] > i) return -1;
  return lo < a.n_seqs ? lo : -1;
}

// The sequence of row i and the place of its token there; b < 0: of none.
struct KvToken {
  int b;
  int64_t place;
};
__device__ __forceinline__ KvToken kv_token(const KvArgs& a, int i) {
  KvToken t{-1, 0};
  if (a.n_seqs < kWave) {  // every offset and length at once: one wait instead of two
    const int lane = threadIdx.x & (kWave - 1);
    const int off = lane <= a.n_seqs ? a.offs[lane] : 0, len = lane < a.n_seqs ? a.lens[lane] : 0;
    t.b = __popcll(__ballot(lane <= a.n_seqs && off <= i)) - 1;
    if (t.b >= a.n_seqs) t.b = -1;
    if (t.b >= 0)
      t.place = (int64_t)__builtin_amdgcn_readlane(len, t.b) - __builtin_amdgcn_readlane(off, t.b + 1) + i;
    return t;
  }
  t.b = kv_sequence_of(a, i);
  if (t.b >= 0) t.place = (int64_t)a.lens[t.b] - a.offs[t.b + 1] + i;
  return t;
}

// Byte offset in the cache of key/value head h of the page that holds place
// p of sequence b, or -1 where there is none.
__device__ __forceinline__ int64_t kv_page_base(const KvArgs& a, int b, int64_t p, int h) {
  if (p < 0 || (p >> a.page_shift) >= a.pages_per_seq) return -1;
  const int page = a.table[(int64_t)b * a.pages_per_seq + (p >> a.page_shift)];
  if ((unsigned)page >= (unsigned)a.n_pages) return -1;
  return ((int64_t)page * a.Hk + h) * a.page_bytes;
}

}  // namespace svr
