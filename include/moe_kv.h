/*
 * moe_kv.h -- C ABI of the attention half of a verify step on a paged 4-bit
 * key/value cache, for AMD Instinct MI355X (gfx950): head norms, position
 * rotation and append in one pass; attention over the cache; reading rows
 * back as values.
 *
 * "Step-5 Preview GGUF" (Model background, configuration table): 64 query
 * heads on 4 key/value heads of size 192, 64 or 192 rotated dimensions, a
 * sliding window of 512 tokens in the window layers; (Runtime support
 * table): attention scale 1/sqrt(192).  "Support Step3.5/3.7 flash mtp3"
 * (Overview, data-flow trace): the verify batch is four rows of one sequence
 * and its rejected tail is overwritten by the next round, which here means:
 * lower seq_lens and append again.
 *
 * BATCH.  A batch is n_seqs sequences with q_offsets[b+1] - q_offsets[b] new
 * rows each, rows of all sequences one after another in q, k, v and out;
 * seq_lens[b] counts the tokens of sequence b WITH its new rows.  Row i of
 * sequence b is the token at place p = seq_lens[b] - q_offsets[b+1] + i.
 * Rows at or behind q_offsets[n_seqs] (padding) are not written; q, k, v and
 * positions have them, with any values.
 * Token p of sequence b lives in page page_table[b][p / page_size], at
 * p % page_size.
 *
 * CACHE LAYOUT.  n_pages pages; page x holds for each key/value head h
 * page_size * (D + D/16) bytes at (x * n_kv_heads + h) * that, D = head_dim:
 *   keys    [page_size][D/2]  two 4-bit codes a byte, the even channel low
 *   values  [page_size][D/2]
 *   key scales   [page_size][D/32]  one byte for 32 channels
 *   value scales [page_size][D/32]
 * A code c stands for (-1)^(c>>3) * {0, 0.5, 1, 1.5, 2, 3, 4, 6}[c & 7], a
 * scale byte e for 2^(e-127) (the microscaling formats E2M1 and E8M0).  A
 * block of 32 values x is stored with the least whole E in [-126, 125] for
 * which max|x| <= 7 * 2^E (0 if all are zero; e = E + 127), and for each x
 * the code nearest to x * 2^-E, the even code between two, at most 6 in
 * size, bit 3 set where x < 0.  So no value is off by more than half of the
 * widest step of its block.  The rotated key is rounded from 64 bits.
 * A token whose key or value holds a NaN or infinity is stored with key
 * scale bytes 255 (NaN) and a value of zeros: every row that attends to it
 * becomes NaN, no other row does.
 *
 * OWNERSHIP, ORDERING, ERRORS.  As in moe_layer.h: every pointer but the two
 * structs is a device pointer of the caller; calls allocate nothing, keep
 * nothing, enqueue on hip_stream and return without synchronising; status
 * codes MOE_OK, MOE_ERR_*.  Nothing is enqueued unless MOE_OK or
 * MOE_ERR_LAUNCH is returned.  Outputs must not alias inputs or each other.
 * The kernels check what only they can see: a token whose page_table entry
 * is outside [0, n_pages), or whose place is negative or beyond the table,
 * is not stored by append, reads back as zeros and is hidden from attention.
 */
#ifndef SVR_MOE_KV_H
#define SVR_MOE_KV_H

#include <stddef.h>
#include <stdint.h>

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* flags of moe_kv_desc */
#define MOE_KV_ROTARY_INTERLEAVED 1 /* rotate neighbours (2j, 2j+1), not (j, j + rotary/2) */

#define MOE_KV_MAX_HEADS 1024
#define MOE_KV_MAX_SEQS 65536
#define MOE_KV_MAX_TOKENS 1048576 /* rows of one call, and tokens of one page table row */

typedef struct moe_kv_desc {
  int32_t n_heads;     /* query heads, a multiple of n_kv_heads, at most MOE_KV_MAX_HEADS */
  int32_t n_kv_heads;  /* key/value heads */
  int32_t head_dim;    /* 64, 128, 192 or 256 */
  int32_t page_size;   /* tokens of a page: a power of two, 16 to 1024 */
  int32_t window;      /* tokens a row sees, itself included; 0: all up to itself */
  int32_t rotary_dims; /* leading channels rotated: a multiple of 16, at most head_dim; 0: none */
  int32_t flags;       /* MOE_KV_ROTARY_INTERLEAVED or 0 */
  float scale;         /* factor of the scores, > 0; 0: 1/sqrt(head_dim) */
  float norm_eps;      /* epsilon of the head norms, >= 0 */
} moe_kv_desc;

typedef struct moe_kv_batch {
  int32_t n_seqs;        /* sequences */
  int32_t n_tokens;      /* rows that q, k, v and out have (padding included) */
  int32_t max_rows;      /* no sequence has more new rows than this (rows above it: see below) */
  int32_t pages_per_seq; /* columns of page_table */
  const int32_t* q_offsets;  /* [n_seqs + 1], ascending, from 0 */
  const int32_t* seq_lens;   /* [n_seqs] */
  const int32_t* page_table; /* [n_seqs][pages_per_seq] */
} moe_kv_batch;

/* Bytes of a cache of n_pages pages, in *bytes.  16-byte aligned caches only. */
int32_t moe_kv_cache_bytes(const moe_kv_desc* desc, int64_t n_pages, int64_t* bytes);

/* Norms, rotation and append, ONE launch.  dtype: MOE_F32, MOE_BF16 or
 * MOE_F16, of q, k, v and q_out.  q [n_tokens][n_heads][D], k and v
 * [n_tokens][n_kv_heads][D] with rows q_stride, k_stride, v_stride elements
 * apart (views of one fused projection need no copy), q_out contiguous [n_tokens][n_heads][D].
 *   q_out = rotate(norm(q) * q_norm), k likewise with k_norm, v as it is;
 *   norm(x) = x / sqrt(mean(x^2) + norm_eps) over a head's D channels;
 *   q_norm, k_norm [D] float, NULL: no norm.
 * rotate turns channel pair j < rotary_dims/2 by pos * inv_freq[j] (float
 * [rotary_dims/2], the angle taken in 64 bits); pos = positions[i] (int32
 * [n_tokens]), or the token's place where positions is NULL.  k and v of
 * row i are stored in the cache at its place.  q and q_out may both be NULL
 * (append only).  Two rows of one call must not share a place in a page.
 * MOE_ERR_NULL: a NULL struct, k, v, cache or batch array, exactly one of q
 * and q_out, rotary_dims > 0 without inv_freq.  MOE_ERR_SHAPE: desc or batch
 * out of range, n_pages < 1, a stride smaller than a row.  MOE_ERR_DTYPE.
 * MOE_ERR_ARG: flags, scale or norm_eps invalid, a pointer not aligned to
 * its elements, cache not 16-byte aligned.  n_tokens == 0 or n_seqs == 0:
 * nothing to do, MOE_OK (after the checks of desc and batch). */
int32_t moe_kv_append(const moe_kv_desc* desc, const moe_kv_batch* batch, int32_t dtype,
                      const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const void* v, int64_t v_stride, const float* q_norm, const float* k_norm,
                      const float* inv_freq, const int32_t* positions, void* cache,
                      int32_t n_pages, void* q_out, void* hip_stream);

/* Device workspace, in *bytes, of moe_kv_attention for this desc and every
 * batch of at most these n_seqs, n_tokens, max_rows and pages_per_seq (the
 * arrays may be NULL), 60 MB at most.  It begins with 16384 bytes of counters,
 * which must be zero before the first call that uses the workspace; every call
 * leaves them zero, so zero-fill a workspace once when it is allocated.  Calls
 * that share one must not overlap in time.  0 is possible, and then workspace
 * may be NULL. */
int32_t moe_kv_attention_workspace_bytes(const moe_kv_desc* desc, const moe_kv_batch* batch,
                                         size_t* bytes);

/* Attention of the batch's new rows over the cache, which must hold them
 * already (append first).  q [n_tokens][n_heads][D] of dtype, rows q_stride
 * elements apart; out contiguous [n_tokens][n_heads][D] of the same type.
 *   s_t = scale * q . key_t for the tokens t a row sees: t <= p, and
 *   t > p - window where window > 0;  out = sum_t softmax(s)_t value_t.
 * Query head h reads key/value head h / (n_heads / n_kv_heads).  A row that
 * sees no token gives zeros.  lse [n_tokens][n_heads] float, may be NULL:
 * the natural log of sum_t e^(s_t) (-inf for a row that sees nothing), with
 * which parts of one attention can be joined.  Rows of a sequence from
 * max_rows on are left unwritten.
 * Keys and values enter exactly; sums are 32-bit; the query enters exactly for
 * MOE_BF16, with 16 bits or more for MOE_F16, 24 for MOE_F32; the softmax weights
 * with 16 bits, 24 for MOE_F32.
 * Errors as moe_kv_append, and MOE_ERR_WORKSPACE for a workspace that is
 * too small, MOE_ERR_ARG for one that is not 256-byte aligned, MOE_ERR_SHAPE
 * for more work than a launch can take: a batch is always served where
 * n_tokens * n_heads / 16 + n_seqs * n_kv_heads is at most 16 million. */
int32_t moe_kv_attention(const moe_kv_desc* desc, const moe_kv_batch* batch, int32_t dtype,
                         const void* q, int64_t q_stride, const void* cache, int32_t n_pages,
                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                         void* hip_stream);

/* The stored keys and values of the batch's rows as float
 * [n_tokens][n_kv_heads][D] (key NaN for a token stored as NaN; zeros where
 * nothing is stored).  k_out or v_out may be NULL.  MOE_ERR_SHAPE where
 * n_tokens * ceil(n_kv_heads * D / 2048) is 2^24 or more. */
int32_t moe_kv_read(const moe_kv_desc* desc, const moe_kv_batch* batch, const void* cache,
                    int32_t n_pages, float* k_out, float* v_out, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SVR_MOE_KV_H */
