// Host side of attention over the paged 4-bit cache (include/moe_kv.h): the
// split of the work, and the kernel that joins the splits of a row.
#include "kv_attention.h"

namespace svr {

extern template int32_t launch_kv_attention<64>(const AttnArgs&, int32_t, int, int, hipStream_t);
extern template int32_t launch_kv_attention<128>(const AttnArgs&, int32_t, int, int, hipStream_t);
extern template int32_t launch_kv_attention<192>(const AttnArgs&, int32_t, int, int, hipStream_t);
extern template int32_t launch_kv_attention<256>(const AttnArgs&, int32_t, int, int, hipStream_t);

namespace {

// One wave a row and head: weighs its splits' sums by their maxima.
template <typename T>
__global__ __launch_bounds__(kBlock) void k_kv_join(AttnArgs a, int row_tiles) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t at = (int64_t)blockIdx.x * kWavesPerBlock + (threadIdx.x >> 6);
  if (at >= (int64_t)a.kv.n_tokens * a.kv.Hq) return;
  const int i = (int)(at / a.kv.Hq), h = (int)(at % a.kv.Hq);
  const int b = kv_sequence_of(a.kv, i);
  if (b < 0) return;
  const KvRows sq = kv_rows(a.kv, b);
  const int m = i - sq.off;
  if (m >= sq.rows) return;
  const int r = m * a.G + h % a.G, r0 = r / (16 * row_tiles) * (16 * row_tiles);
  const int r_last = min(sq.rows * a.G, r0 + 16 * row_tiles) - 1;
  const KvRange rg = kv_range(a.kv, sq.len, sq.place0 + r0 / a.G, sq.place0 + r_last / a.G, a.splits,
                              a.min_tiles);
  if (rg.used == 1) return;
  const float2* ml = a.part_ml + at * a.splits;
  float M = -INFINITY;
  for (int s = 0; s < rg.used; ++s) M = fmaxf(M, ml[s].x);
  float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const int n = a.kv.D / kWave;
  for (int s = 0; s < rg.used; ++s) {
    const float2 x = ml[s];
    const float w = x.x == M ? 1.f : __builtin_amdgcn_exp2f(x.x - M);
    L += w * x.y;
    const float* p = a.part_o + (at * a.splits + s) * a.kv.D + lane;
    for (int j = 0; j < n; ++j) o[j] += w * p[kWave * j];
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  for (int j = 0; j < n; ++j) ((T*)a.out)[at * a.kv.D + lane + kWave * j] = (T)(o[j] * inv);
  if (a.lse && lane == 0)
    a.lse[at] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * 0.6931471805599453f;
}

// How a batch is cut: by its sizes alone (the lengths are on the device).
struct AttnPlan {
  int row_tiles, tiles, splits, min_tiles;
  int64_t grid;
  size_t o_bytes, bytes;
};

AttnPlan attn_plan(const moe_kv_desc* d, const moe_kv_batch* b, int32_t dtype) {
  AttnPlan p{};
  const int G = d->n_heads / d->n_kv_heads;
  const int64_t rows = (int64_t)(b->max_rows < b->n_tokens ? b->max_rows : b->n_tokens) * G;
  p.row_tiles = attn_row_tiles(rows, d->head_dim, dtype);
  p.tiles = (int)((rows + 16 * p.row_tiles - 1) / (16 * p.row_tiles));
  p.min_tiles = kAttnWaves;  // a tile a wave
  const int64_t base = (int64_t)b->n_seqs * d->n_kv_heads * p.tiles;
  int64_t seen = (int64_t)b->pages_per_seq * d->page_size;
  if (d->window && d->window + (int64_t)b->max_rows < seen) seen = d->window + (int64_t)b->max_rows;
  const int64_t most = (seen / kAttnTile + 2 + p.min_tiles - 1) / p.min_tiles;
  int64_t s = base > 0 ? 512 / base : 1;
  s = s < 1 ? 1 : s;
  p.splits = (int)(s < most ? s : most);
  p.grid = base * p.splits;
  if (p.splits > 1) {
    const size_t n = (size_t)b->n_tokens * d->n_heads * p.splits;
    p.o_bytes = (n * d->head_dim * 4 + 255) & ~(size_t)255;
    p.bytes = p.o_bytes + n * 8;
  }
  return p;
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
  for (int32_t t : {MOE_F32, MOE_BF16}) {
    const size_t n = attn_plan(desc, batch, t).bytes;
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
  if (p.grid > INT32_MAX) return MOE_ERR_SHAPE;
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
  a.part_o = (float*)workspace;
  a.part_ml = (float2*)((uint8_t*)workspace + p.o_bytes);
  a.c = (desc->scale > 0.f ? desc->scale : 1.f / sqrtf((float)desc->head_dim)) * 1.4426950408889634f;
  a.G = desc->n_heads / desc->n_kv_heads;
  a.tiles = p.tiles;
  a.splits = p.splits;
  a.min_tiles = p.min_tiles;
  a.vec = (uintptr_t)q % 16 == 0 && q_stride * es % 16 == 0 ? 1 : 0;
  hipStream_t st = (hipStream_t)hip_stream;
  (void)hipGetLastError();
  switch (desc->head_dim) {
    case 64: rc = launch_kv_attention<64>(a, dtype, p.row_tiles, (int)p.grid, st); break;
    case 128: rc = launch_kv_attention<128>(a, dtype, p.row_tiles, (int)p.grid, st); break;
    case 192: rc = launch_kv_attention<192>(a, dtype, p.row_tiles, (int)p.grid, st); break;
    default: rc = launch_kv_attention<256>(a, dtype, p.row_tiles, (int)p.grid, st); break;
  }
  if (rc != MOE_OK || p.splits == 1) return rc;
  const int64_t n = (int64_t)batch->n_tokens * desc->n_heads;
  const dim3 g((unsigned)((n + kWavesPerBlock - 1) / kWavesPerBlock)), t(kBlock);
  switch (dtype) {
    case MOE_F32: hipLaunchKernelGGL(k_kv_join<float>, g, t, 0, st, a, p.row_tiles); break;
    case MOE_BF16: hipLaunchKernelGGL(k_kv_join<bf16>, g, t, 0, st, a, p.row_tiles); break;
    default: hipLaunchKernelGGL(k_kv_join<_Float16>, g, t, 0, st, a, p.row_tiles); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
