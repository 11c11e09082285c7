// Host side of attention over the paged 4-bit cache (include/moe_kv.h): the
// split of the work, and the kernel that joins the splits of a row.
#include "kv_attention.h"

namespace svr {

extern template int32_t launch_kv_attention<64>(const AttnArgs&, int32_t, int, int, int, hipStream_t);
extern template int32_t launch_kv_attention<128>(const AttnArgs&, int32_t, int, int, int, hipStream_t);
extern template int32_t launch_kv_attention<192>(const AttnArgs&, int32_t, int, int, int, hipStream_t);
extern template int32_t launch_kv_attention<256>(const AttnArgs&, int32_t, int, int, int, hipStream_t);

namespace {

constexpr int kMaxSplits = 128;

// Joins the splits of one row and head: out = sum_s w_s O_s / sum_s w_s l_s
// with w_s = 2^(m_s - max m).  One workgroup a row and head; a slot of D/4
// lanes reads a split's sums 16 bytes a lane, the slots take the splits in
// turn.  Bound by latency, not bytes (a row's parts are at most 128 KB): the
// first kBatch of a slot's reads are issued before it is known which splits
// are in use (the workspace holds them all, what is not in use is dropped).
// Rows for at most a workgroup a CU: all reads at once, by 512 threads (1 row
// of 64 heads with 128 splits 5.1 us, 8.2 with 256 threads; 4 rows with 32 5.0
// us).  More: one read, by 256 (12 rows of 64 heads with 20 of 43 splits in use
// 5.7 us, 9.9 with all at once).
template <int D, int kThreads, int kBatch, typename T>
__global__ __launch_bounds__(kThreads) void k_kv_join(AttnArgs a) {
  constexpr int L = D / 4, kSlots = kThreads / L;
  __shared__ float s_w[kMaxSplits];
  __shared__ f32x4v s_o[kSlots][L];
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t at = blockIdx.x;  // of the parts
  const int slot = threadIdx.x / L, c = threadIdx.x % L;
  const int splits = a.splits.d;
  const float2* ml = a.part_ml + at * splits;
  const f32x4v* part = reinterpret_cast<const f32x4v*>(a.part_o + at * splits * D) + c;
  float2 x[kMaxSplits / kWave];
#pragma unroll
  for (int j = 0; j < kMaxSplits / kWave; ++j) x[j] = ml[min(lane + kWave * j, splits - 1)];
  f32x4v v[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) v[j] = part[(int64_t)min(slot + kSlots * j, splits - 1) * L];

  const int kvh = a.G.of(blockIdx.x), row = a.heads.of(kvh);  // at = (row Hk + head) G + query of the head
  const int per = kv_per(a, kv_lane_rows(a, lane)), b = a.by_seq ? a.rows.of(row) : kv_sequence_of(a.kv, row);
  if (b < 0) return;
  const KvRows sq = kv_rows(a.kv, b);
  const int m = a.by_seq ? row - b * a.kv.max_rows : row - sq.off;
  if (m >= sq.rows) return;
  const int span = 16 * a.row_tiles, G = a.G.d;
  const int r0 = (m * G + (int)blockIdx.x - kvh * G) & ~(span - 1);
  const int r_last = min(sq.rows * G, r0 + span) - 1;
  const KvRange rg = kv_range(a, sq.len, sq.place0 + a.G.of(r0), sq.place0 + a.G.of(r_last), per);
  if (rg.whole()) return;  // written already
  float M = -INFINITY, sum = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxSplits / kWave; ++j)
    if (rg.uses(lane + kWave * j)) M = fmaxf(M, x[j].x);
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) M = fmaxf(M, __shfl_xor(M, o, kWave));
#pragma unroll
  for (int j = 0; j < kMaxSplits / kWave; ++j)
    if (rg.uses(lane + kWave * j)) {
      const float w = x[j].x == M ? 1.f : __builtin_amdgcn_exp2f(x[j].x - M);
      sum += w * x[j].y;
      if (threadIdx.x < kWave) s_w[lane + kWave * j] = w;
    }
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) sum += __shfl_xor(sum, o, kWave);
  __syncthreads();
  f32x4v acc = {0.f, 0.f, 0.f, 0.f};
  if (slot < kSlots) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int s = slot + kSlots * j;
      if (rg.uses(s)) acc += s_w[s] * v[j];
    }
#pragma unroll 4
    for (int s = slot + kSlots * kBatch; rg.uses(s); s += kSlots) acc += s_w[s] * part[(int64_t)s * L];
    s_o[slot][c] = acc;
  }
  __syncthreads();
  if (slot != 0) return;
#pragma unroll
  for (int j = 1; j < kSlots; ++j) acc += s_o[j][c];
  acc *= sum == 0.f ? 0.f : 1.f / sum;
  const int64_t to = (int64_t)(sq.off + m) * a.kv.Hq + (at - (int64_t)row * a.kv.Hq);
  store4((T*)a.out + to * D + 4 * c, acc);
  if (a.lse && c == 0)
    a.lse[to] = sum == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

template <int D, int kThreads, int kBatch>
void launch_kv_join(const AttnArgs& a, int32_t dtype, unsigned n, hipStream_t st) {
  const dim3 g(n), t(kThreads);
  switch (dtype) {
    case MOE_F32: hipLaunchKernelGGL((k_kv_join<D, kThreads, kBatch, float>), g, t, 0, st, a); break;
    case MOE_BF16: hipLaunchKernelGGL((k_kv_join<D, kThreads, kBatch, bf16>), g, t, 0, st, a); break;
    default: hipLaunchKernelGGL((k_kv_join<D, kThreads, kBatch, _Float16>), g, t, 0, st, a); break;
  }
}
// n: rows x heads.
template <int D>
void launch_kv_join(const AttnArgs& a, int32_t dtype, unsigned n, hipStream_t st) {
  constexpr int kFew = 512, kSlots = kFew / (D / 4);
  if (n <= 256) launch_kv_join<D, kFew, (kMaxSplits + kSlots - 1) / kSlots>(a, dtype, n, st);
  else launch_kv_join<D, 256, 1>(a, dtype, n, st);
}

// How a batch is cut, as far as its sizes say (the lengths are on the device).
struct AttnPlan {
  int row_tiles, tiles, waves, splits, min_tiles, share, group, by_seq, search, first, extra;
  bool join_here;
  int64_t part_rows;
  int64_t grid;
  size_t o_bytes, bytes;
};

// Tiles that a row can see by the batch's table and window.
int64_t attn_seen_tiles(const moe_kv_desc* d, const moe_kv_batch* b) {
  int64_t seen = (int64_t)b->pages_per_seq * d->page_size;
  if (d->window && d->window + (int64_t)b->max_rows < seen) seen = d->window + (int64_t)b->max_rows;
  return seen / kAttnTile + 2;
}

// The plan for workgroups of p.waves: the splits of `all` row tiles of a head.
// Returns whether row tiles are few, and tables long, enough for four splits
// or more and as many as there is room for.
bool attn_split(AttnPlan& p, const moe_kv_desc* d, const moe_kv_batch* b, int32_t dtype, int64_t all) {
  // A part is a tile a wave at least, and as many more for every 64 sequences
  // behind the first, which a workgroup passes over to find it.
  p.min_tiles = p.waves * (1 + (b->n_seqs - 1) / kWave);
  // Work of a head that runs at once.
  const int resident = attn_waves(d->head_dim, p.row_tiles, attn_terms(dtype)) * kAttnWaves / p.waves;
  const int slots = 256 * resident / d->n_kv_heads;
  // Every row tile has one part that is half full on the average.  Where two of
  // each are more than run at once, even sequences are not cut: 97 of 2000
  // tokens 35 us (46 in halves), and longer ones into parts of the mean.
  int64_t share = slots - all / 2;
  if (2 * all > slots && share > all) share = all;
  p.share = (int)(share > slots / 2 ? share : slots / 2);
  p.share = p.share > 0 ? p.share : 1;
  const int64_t tiles = attn_seen_tiles(d, b), most = (tiles + p.min_tiles - 1) / p.min_tiles;
  if (b->n_seqs == 1) {
    const int64_t s = 2 * all > slots ? 1 : slots / all;
    p.splits = (int)(s < kMaxSplits ? s : kMaxSplits);
  } else {
    // Several sequences get up to four times their even part, and sixteen at
    // least: how many are in use goes by the lengths, and a batch of even ones
    // is not cut where there are as many as run at once.  One sequence of 60000
    // tokens among 127 of up to 3000: 69 us, 523 if it is not cut.
    const int64_t s = (4 * (int64_t)slots + all - 1) / all;
    p.splits = tiles <= 3 * p.min_tiles ? 1 : s < kJoinHere ? kJoinHere : s < kMaxSplits ? (int)s : kMaxSplits;
  }
  const bool room = p.splits > 1 && p.splits <= most;
  p.splits = p.splits < most ? p.splits : (int)most;
  return slots / all >= 4 && room;
}

AttnPlan attn_plan(const moe_kv_desc* d, const moe_kv_batch* b, int32_t dtype) {
  AttnPlan p{};
  if (b->n_seqs == 0 || b->n_tokens == 0 || b->max_rows == 0) return p;
  const int G = d->n_heads / d->n_kv_heads;
  const int64_t rows = (int64_t)(b->max_rows < b->n_tokens ? b->max_rows : b->n_tokens) * G;
  p.row_tiles = attn_row_tiles(rows, d->head_dim, dtype);
  const int span = 16 * p.row_tiles;
  p.tiles = (int)((rows + span - 1) / span);
  int64_t all = (int64_t)b->n_seqs * p.tiles;
  const int64_t dense = (int64_t)b->n_tokens * G / span + b->n_seqs;  // see kv_first_tile
  p.search = all > dense;
  all = p.search ? dense : all;
  // Larger workgroups make fewer parts: 4 rows over 60000 tokens 34.7 us (37.2
  // with four waves), 15000 tokens 21.8 (24.2); but a part of 64 rows over
  // 16384, of which there are two, takes 114 us (101), 4 rows over 4000 tokens
  // 26.0 (15.3).
  p.waves = kAttnPartWaves;
  if (p.row_tiles != 2 || !attn_split(p, d, b, dtype, all)) {
    p.waves = kAttnWaves;
    attn_split(p, d, b, dtype, all);
  }
  p.group = p.tiles < 64 ? p.tiles : 64;
  p.first = (int)all;
  p.extra = p.splits == 1 ? 0 : b->n_seqs == 1 ? (int)all * (p.splits - 1) : p.share;
  p.grid = ((all + p.extra + p.group - 1) / p.group * d->n_kv_heads + 7) / 8 * 8 * p.group;
  const int64_t most_rows = (int64_t)b->n_seqs * b->max_rows;
  p.by_seq = most_rows < b->n_tokens;
  p.part_rows = p.by_seq ? most_rows : b->n_tokens;
  if (p.splits > 1) {
    p.join_here = p.splits <= kJoinHere;
    const int first = b->n_seqs == 1 ? (int)all : p.extra;  // first parts lie as the ones behind them do
    const size_t n = p.join_here ? (size_t)(p.extra + first) * d->n_kv_heads * span
                                 : (size_t)p.part_rows * d->n_heads * p.splits;
    p.o_bytes = (n * d->head_dim * 4 + 255) & ~(size_t)255;
    p.bytes = kAttnCounters * sizeof(unsigned) + p.o_bytes + n * 8;
  }
  return p;
}

// What the plan of any batch of up to these sizes needs.  Row tiles times
// splits are at most what runs at once for one sequence, 4 1/4 of that for
// several (at most a quarter of it row tiles, each with a part too many); where
// the last workgroup joins, twice p.share, which is at most what runs at once.
size_t attn_most_bytes(const moe_kv_desc* d, const moe_kv_batch* b, int32_t dtype) {
  if (b->n_seqs == 0 || b->n_tokens == 0 || b->max_rows == 0) return 0;
  if (attn_seen_tiles(d, b) <= kAttnWaves) return 0;  // never cut
  const int64_t rows = (int64_t)(b->max_rows < b->n_tokens ? b->max_rows : b->n_tokens) *
                       (d->n_heads / d->n_kv_heads);
  size_t most = 0;
  for (int rt = 1; rt <= attn_row_tiles(rows, d->head_dim, dtype); ++rt) {
    const int slots = 256 * attn_waves(d->head_dim, rt, attn_terms(dtype)) / d->n_kv_heads;
    const int parts = b->n_seqs == 1 ? slots : slots < 1 ? 2 : 4 * slots + slots / 4;
    const size_t n = (size_t)parts * d->n_kv_heads * 16 * rt;
    const size_t bytes = kAttnCounters * sizeof(unsigned) + ((n * d->head_dim * 4 + 255) & ~(size_t)255) + n * 8;
    most = bytes > most ? bytes : most;
  }
  return most;
}

}  // namespace
}  // namespace svr

using namespace svr;

extern "C" {

int32_t moe_kv_attention_workspace_bytes(const moe_kv_desc* desc, const moe_kv_batch* batch,
                                         size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  int32_t rc = kv_check_desc(desc);
  if (rc == MOE_OK) rc = kv_check_batch(desc, batch, false);
  if (rc != MOE_OK) return rc;
  size_t most = 0;
  for (int32_t t : {MOE_F32, MOE_BF16, MOE_F16}) {
    const size_t n = attn_most_bytes(desc, batch, t);
    most = n > most ? n : most;
  }
  *bytes = most;
  return MOE_OK;
}

int32_t moe_kv_attention(const moe_kv_desc* desc, const moe_kv_batch* batch, int32_t dtype,
                         const void* q, int64_t q_stride, const void* cache, int32_t n_pages,
                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                         void* hip_stream) {
  int32_t rc = kv_check_desc(desc);
  if (rc == MOE_OK) rc = kv_check_batch(desc, batch, true);
  if (rc != MOE_OK) return rc;
  const int es = kv_elem_size(dtype);
  if (!es) return MOE_ERR_DTYPE;
  if (n_pages < 1) return MOE_ERR_SHAPE;
  if (batch->n_tokens == 0 || batch->n_seqs == 0 || batch->max_rows == 0) return MOE_OK;
  if (!q || !cache || !out) return MOE_ERR_NULL;
  if (q_stride < (int64_t)desc->n_heads * desc->head_dim) return MOE_ERR_SHAPE;
  if (((uintptr_t)q | (uintptr_t)out) % es || (uintptr_t)lse % 4 || (uintptr_t)cache % 16)
    return MOE_ERR_ARG;
  const AttnPlan p = attn_plan(desc, batch, dtype);
  if (!kv_grid_fits(p.grid, p.waves * kWave)) return MOE_ERR_SHAPE;
  if (p.bytes) {
    if (!workspace) return MOE_ERR_NULL;
    if (workspace_bytes < p.bytes) return MOE_ERR_WORKSPACE;
    if ((uintptr_t)workspace % 256) return MOE_ERR_ARG;
  }

  AttnArgs a{};
  a.kv = kv_args(desc, batch, n_pages);
  a.q = q;
  a.qs = q_stride;
  a.cache = (const uint8_t*)cache;
  a.out = out;
  a.lse = lse;
  a.ctr = p.join_here ? (unsigned*)workspace : nullptr;
  a.part_o = (float*)workspace + kAttnCounters;
  a.part_ml = (float2*)((uint8_t*)a.part_o + p.o_bytes);
  a.c = (desc->scale > 0.f ? desc->scale : 1.f / sqrtf((float)desc->head_dim)) * 1.4426950408889634f;
  a.G = make_divider(desc->n_heads / desc->n_kv_heads);
  a.tiles = make_divider(p.tiles);
  a.splits = make_divider(p.splits);
  a.heads = make_divider(desc->n_kv_heads);
  a.share = make_divider(p.share);
  a.group = make_divider(p.group);
  a.min_tiles = p.min_tiles;
  a.row_tiles = p.row_tiles;
  a.by_seq = p.by_seq;
  a.search = p.search;
  a.first = p.first;
  a.extra = p.extra;
  a.rows = make_divider(batch->max_rows);
  hipStream_t st = (hipStream_t)hip_stream;
  (void)hipGetLastError();
  switch (desc->head_dim) {
    case 64: rc = launch_kv_attention<64>(a, dtype, p.row_tiles, p.waves, (int)p.grid, st); break;
    case 128: rc = launch_kv_attention<128>(a, dtype, p.row_tiles, p.waves, (int)p.grid, st); break;
    case 192: rc = launch_kv_attention<192>(a, dtype, p.row_tiles, p.waves, (int)p.grid, st); break;
    default: rc = launch_kv_attention<256>(a, dtype, p.row_tiles, p.waves, (int)p.grid, st); break;
  }
  if (rc != MOE_OK || p.splits == 1 || p.join_here) return rc;
  const unsigned n = (unsigned)p.part_rows * (unsigned)desc->n_heads;
  switch (desc->head_dim) {
    case 64: launch_kv_join<64>(a, dtype, n, st); break;
    case 128: launch_kv_join<128>(a, dtype, n, st); break;
    case 192: launch_kv_join<192>(a, dtype, n, st); break;
    default: launch_kv_join<256>(a, dtype, n, st); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
