// Host side of attention over the paged 4-bit cache (include/moe_kv.h, and
// with rows of a tree include/moe_tree.h): the
// split of the work, and the kernel that joins the splits of a row.
#include "kv_attention.h"
#include "tree.h"

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
  const KvRange rg = a.mask ? kv_tree_range(a, sq, per)
                            : kv_range(a, sq.len, sq.place0 + a.G.of(r0), sq.place0 + a.G.of(r_last), per);
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
  int row_tiles, tiles, waves, splits, min_tiles, even_tiles, share, group, by_seq, search, first, extra;
  bool join_here;
  int64_t part_rows;
  int64_t cost;  // of one tree's parts
  int64_t grid;
  size_t o_bytes, bytes;
};

// Tiles that a row can see by the batch's table and window.
int64_t attn_seen_tiles(const moe_kv_desc* d, const moe_kv_batch* b) {
  int64_t seen = (int64_t)b->pages_per_seq * d->page_size;
  if (d->window && d->window + (int64_t)b->max_rows < seen) seen = d->window + (int64_t)b->max_rows;
  return seen / kAttnTile + 2;
}

// Workgroups of a CU, and a head's row tiles or parts that run at once.
int attn_resident(const moe_kv_desc* d, int row_tiles, int32_t dtype, int waves) {
  return attn_waves(d->head_dim, row_tiles, attn_terms(dtype)) * kAttnWaves / waves;
}
int attn_slots(const moe_kv_desc* d, int row_tiles, int32_t dtype, int waves) {
  return 256 * attn_resident(d, row_tiles, dtype, waves) / d->n_kv_heads;
}

// Splits of one tree's row tiles, which see the same tokens, so that parts are
// alike, and what they cost, in tiles: those of a part, and what it costs to
// begin and to join.  Row tiles of a head and a split are one group, groups go
// round the XCDs (see the kernel).  An XCD with one group more than it has room
// for takes a second round, whose row tiles no longer read the same tokens at the
// same time: 24 rows over 40000 tokens, 4 heads, eight waves 101 us with four
// splits, 146 with five to ten.
//   More parts than run at once fill the rounds of row tiles of which few fit: 65
// rows of 64 heads on 4 over 60000 tokens, bf16, D = 192 (33 row tiles, room for
// 128) 319 us with ten, 478 with two.  They have twelve steps a wave at least (65
// rows of 128 heads on 8, fp16, 65 row tiles and room for 64: over 2000 tokens 54
// us, 60 in thirds; over 3500 82, 77 in halves), and are up to three times what
// runs at once (with four times, in thirds, 327 us over 20000 tokens instead of 343;
// uncut 419).  Row tiles that pass what runs at once by more than a quarter fill
// about half of a round, which takes half the time: not cut (96 of those rows over
// 3500 tokens 84 us, 90 in halves).
constexpr int kTreeSteps = 12;
struct TreeSplits {
  int splits;
  int64_t cost;
};
// The most parts of one tree, in what runs at once: row tiles of which eight or
// more fit waste little of it, and need the workspace that they need without masks.
int64_t tree_rounds(int64_t row_tiles, int64_t at_once) { return 8 * row_tiles < at_once ? 1 : 3; }
TreeSplits tree_splits(int64_t row_tiles, int heads, int resident, int64_t tiles, int min_tiles, int64_t at_once,
                       int64_t most_parts, int step) {
  const int64_t group = row_tiles < 64 ? row_tiles : 64, room = 256 / 8 * resident;  // workgroups of an XCD at once
  TreeSplits best{1, 0};
  for (int s = 1; s <= kMaxSplits && (s - 1) * min_tiles < tiles && row_tiles * s <= most_parts; ++s) {
    if (s > 1 && row_tiles * s > at_once && (tiles < (int64_t)kTreeSteps * step * s || 4 * row_tiles > 5 * at_once)) break;
    const int64_t groups = (row_tiles * s + group - 1) / group * heads;
    const int64_t rounds = ((groups + 7) / 8 * group + room - 1) / room;
    int64_t cost = (tiles + s - 1) / s;
    cost = cost > min_tiles ? cost : min_tiles;
    if (rounds > 1) cost = rounds * (cost * 8 / 5 + 12);
    cost += 12 + (s > 1 ? 8 : 0) + (s > kJoinHere ? 8 : 0);
    if (s == 1 || cost < best.cost) best = TreeSplits{s, cost};
  }
  return best;
}

// The plan for workgroups of p.waves: the splits of `all` row tiles of a head.
// Returns whether row tiles are few, and tables long, enough for four splits
// or more and as many as there is room for.
bool attn_split(AttnPlan& p, const moe_kv_desc* d, const moe_kv_batch* b, int32_t dtype, int64_t all, bool tree) {
  p.even_tiles = kWholeRange;
  // A part is a tile a wave at least, and as many more for every 64 sequences
  // behind the first, which a workgroup passes over to find it.
  p.min_tiles = p.waves * (1 + (b->n_seqs - 1) / kWave);
  // Trees of few rows: two, since joining takes as long as a step (13 rows over
  // 777 tokens 11.2 us, 12.4 with one, 13.6 with three; fp32, a window of 512
  // 18.8 and 23.6).
  if (tree && p.row_tiles == 1) p.min_tiles *= 2;
  const int resident = attn_resident(d, p.row_tiles, dtype, p.waves), slots = attn_slots(d, p.row_tiles, dtype, p.waves);
  // Every row tile has one part that is half full on the average.  Where two of
  // each are more than run at once, even sequences are not cut: 97 of 2000
  // tokens 35 us (46 in halves), and longer ones into parts of the mean.
  int64_t share = slots - all / 2;
  if (2 * all > slots && share > all) share = all;
  p.share = (int)(share > slots / 2 ? share : slots / 2);
  // Trees have work for longer parts than single rows do, and more of them on the
  // average than run at once: parts of the mean however many row tiles there are
  // (up to twice what runs at once, by the workspace), eight steps a wave at
  // least (29 trees of up to 26 rows over 5000 tokens, fp16, 75 us, 82 without; 40
  // of up to 7 over 20000 198 and 241; with one step at least 60 of up to 10 over
  // 3000 54 us, 48 with eight).  Even trees are not cut, as before.
  if (tree && b->n_seqs == 1) p.share = slots;  // as even (61 rows over 60000 tokens 256 us, 275 without)
  if (tree && b->n_seqs > 1 && 2 * all > slots) {
    p.share = (int)(all < 2 * slots ? all : 2 * slots);
    p.min_tiles = p.min_tiles > 8 * p.waves ? p.min_tiles : 8 * p.waves;
  }
  p.share = p.share > 0 ? p.share : 1;
  const int64_t tiles = attn_seen_tiles(d, b), most = (tiles + p.min_tiles - 1) / p.min_tiles;
  if (tree && b->n_seqs == 1) {
    const int64_t rounds = tree_rounds(all, attn_slots(d, p.row_tiles, dtype, kAttnWaves));
    const TreeSplits t = tree_splits(all, d->n_kv_heads, resident, tiles, p.min_tiles, slots, slots * rounds, p.waves);
    p.splits = t.splits;
    // By the length, which the table may pass by far: parts of fewer steps are as many
    // as run at once, by share (65 rows of 64 heads on 4 over 2000 tokens in a table
    // of 60000 36 us, 46 in all splits; over 20000 127, 153 by share).
    p.even_tiles = kTreeSteps * p.waves;
    p.cost = t.cost;
  } else if (b->n_seqs == 1) {
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

AttnPlan attn_plan(const moe_kv_desc* d, const moe_kv_batch* b, int32_t dtype, bool tree) {
  AttnPlan p{};
  if (b->n_seqs == 0 || b->n_tokens == 0 || b->max_rows == 0) return p;
  const int G = d->n_heads / d->n_kv_heads;
  const int64_t rows = (int64_t)(b->max_rows < b->n_tokens ? b->max_rows : b->n_tokens) * G;
  p.row_tiles = attn_row_tiles(rows, d->head_dim, dtype);
  // Trees of which a wave has two or three steps of 16 rows in all, as far as the
  // table says: their time is one step after another, which is shorter for one
  // row tile (7 rows over 777 tokens 10.5 us, 15.2 with two; 13 over 10000 28 and
  // 42; but 7 over 40000 49 and 45, 32 over 10000 42 and 36).
  if (tree && (int64_t)b->n_seqs * ((rows + 15) / 16) * d->n_kv_heads * attn_seen_tiles(d, b) <= 8192)
    p.row_tiles = 1;
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
  const bool large = p.row_tiles == 2 && attn_split(p, d, b, dtype, all, tree);
  const AttnPlan parts = p;
  p.waves = kAttnWaves;
  if (!large || (tree && b->n_seqs == 1)) attn_split(p, d, b, dtype, all, tree);
  // (One tree: those that cost less, of which the larger take a tile in half the time.)
  if (large && (!tree || b->n_seqs > 1 || parts.cost <= 2 * p.cost)) p = parts;
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
// splits are at most what runs at once for one sequence, three times that for one
// tree of more than a few row tiles, 4 1/4 for several sequences (at most a quarter
// of it row tiles, each with a part too many); where the last workgroup joins, twice
// p.share, which is at most what runs at once, of trees twice that.
size_t attn_most_bytes(const moe_kv_desc* d, const moe_kv_batch* b, int32_t dtype) {
  if (b->n_seqs == 0 || b->n_tokens == 0 || b->max_rows == 0) return 0;
  if (attn_seen_tiles(d, b) <= kAttnWaves) return 0;  // never cut
  const int64_t rows = (int64_t)(b->max_rows < b->n_tokens ? b->max_rows : b->n_tokens) *
                       (d->n_heads / d->n_kv_heads);
  size_t most = 0;
  for (int rt = 1; rt <= attn_row_tiles(rows, d->head_dim, dtype); ++rt) {
    const int slots = attn_slots(d, rt, dtype, kAttnWaves);
    const int64_t parts = b->n_seqs == 1 ? slots * tree_rounds((rows + 16 * rt - 1) / (16 * rt), slots)
                          : slots < 1    ? 2
                                         : 4 * slots + slots / 4;
    const size_t n = (size_t)parts * d->n_kv_heads * 16 * rt;
    const size_t bytes = kAttnCounters * sizeof(unsigned) + ((n * d->head_dim * 4 + 255) & ~(size_t)255) + n * 8;
    most = bytes > most ? bytes : most;
  }
  return most;
}

// Attention of a batch's rows; mask: those of a tree (NULL: each sees the ones before it).
int32_t attention(const moe_kv_desc* desc, const moe_kv_batch* batch, int32_t dtype, const uint64_t* mask,
                  int32_t mask_words, const void* q, int64_t q_stride, const void* cache, int32_t n_pages,
                  void* out, float* lse, void* workspace, size_t workspace_bytes, void* hip_stream) {
  const int es = kv_elem_size(dtype);
  if (!es) return MOE_ERR_DTYPE;
  if (n_pages < 1) return MOE_ERR_SHAPE;
  if (batch->n_tokens == 0 || batch->n_seqs == 0 || batch->max_rows == 0) return MOE_OK;
  if (!q || !cache || !out) return MOE_ERR_NULL;
  if (q_stride < (int64_t)desc->n_heads * desc->head_dim) return MOE_ERR_SHAPE;
  if (((uintptr_t)q | (uintptr_t)out) % es || (uintptr_t)lse % 4 || (uintptr_t)cache % 16)
    return MOE_ERR_ARG;
  const AttnPlan p = attn_plan(desc, batch, dtype, mask != nullptr);
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
  a.even_tiles = p.even_tiles;
  a.row_tiles = p.row_tiles;
  // Rows of a tile: whole tokens, and one cut at either end; those of a tree: all of them.
  a.reach = a.kv.window + (mask ? batch->max_rows : 16 * p.row_tiles / a.G.d) + 2 + kAttnTile;
  a.mask = reinterpret_cast<const uint32_t*>(mask);
  a.mask_words = 2 * mask_words;
  a.by_seq = p.by_seq;
  a.search = p.search;
  a.first = p.first;
  a.extra = p.extra;
  a.rows = make_divider(batch->max_rows);
  hipStream_t st = (hipStream_t)hip_stream;
  (void)hipGetLastError();
  int32_t rc;
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
  return attention(desc, batch, dtype, nullptr, 0, q, q_stride, cache, n_pages, out, lse, workspace,
                   workspace_bytes, hip_stream);
}

int32_t moe_kv_tree_attention(const moe_kv_desc* desc, const moe_kv_batch* batch, int32_t dtype,
                              const uint64_t* mask, int32_t mask_words, const void* q,
                              int64_t q_stride, const void* cache, int32_t n_pages, void* out,
                              float* lse, void* workspace, size_t workspace_bytes,
                              void* hip_stream) {
  int32_t rc = kv_check_desc(desc);
  if (rc == MOE_OK) rc = kv_check_batch(desc, batch, true);
  if (rc != MOE_OK) return rc;
  if (mask_words < 1 || mask_words > MOE_TREE_MAX_ROWS / 64 || batch->max_rows > 64 * mask_words)
    return MOE_ERR_SHAPE;
  if (batch->n_tokens > 0 && batch->n_seqs > 0 && batch->max_rows > 0 && !mask) return MOE_ERR_NULL;
  if ((uintptr_t)mask % 8) return MOE_ERR_ARG;
  return attention(desc, batch, dtype, mask, mask_words, q, q_stride, cache, n_pages, out, lse,
                   workspace, workspace_bytes, hip_stream);
}

}  // extern "C"
