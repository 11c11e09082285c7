// Sampled verification of drafted tokens (include/moe_sample.h).
//
// Every row of logits is read once, whole rows side by side: which rows the
// accepted path takes is not known before their sums are.  A wave takes tiles
// of 1024 columns, 16 a lane, and leaves for each tile its maximum m and
// z = sum e^((x - m) / T); the last workgroup of a row joins these and tries the
// row's children; the last row of a sequence follows the path, finds the tile
// of its last row in which the cumulative sum passes sample_u, and the column
// in it.
//   Weights are 64-bit: a column weighs 1e-6 of a row, so a cumulative sum of
// 32 bits would give another token one time in a hundred.  2^t for t <= 0 is
// a power of two times its Taylor sum on [-1/2, 1/2] (to (t ln 2)^11 / 11!: the
// rest is below 7e-15); 64-bit products and sums run at the rate of 32-bit ones
// here.
//   Given drafts: a row's children are left out of its tiles' sums and weighed
// one by one.  At the row where the path ends all of them are rejected, so the
// tiles' sums are those of what is left, with nothing subtracted; one launch.
//   Drawn drafts: sums of (p - c q)+ need the row's sum first, and after k
// rejections the sum for k - 1: a launch for each child a row can have, which
// passes over the rows that are undecided and that the path can still reach.
#include <hip/hip_runtime.h>

#include "kv.h"
#include "moe_sample.h"
#include "row_tile.h"
#include "tree.h"

namespace svr {
namespace {

constexpr size_t kSampleCounterBytes = 2 * MOE_SAMPLE_MAX_ROWS * sizeof(unsigned);
constexpr int kSampleSpread = 2048;  // workgroups of a call that are wanted

struct SampleArgs {
  TreeArgs tree;
  const void* x;
  int64_t stride;
  int V, tiles, blocks, tiles_per_block;
  const int32_t* tokens;
  const float* q;  // NULL: given drafts
  int64_t q_stride;
  const float *temp, *accept_u, *sample_u, *vh;
  int hdim;
  int32_t *accepted, *path, *n_acc;
  float* pending;
  unsigned *row_ctr, *seq_ctr;
  uint64_t* info;  // [row][kInfo]
  double* tz;      // [row][tile] sums, relative to the tile's maximum or of (p - c q)+
  float* tm;       // [row][tile] maxima
  int last;        // the launch that ends the call
};

// What a row's last workgroup finds, five words: the sum z relative to its
// maximum, c and S of the drafts rejected so far, the maximum and a token
// (greedy: the largest; given drafts with nothing else left: the best of them),
// the accepted child and how many were tried.
constexpr int kInfo = 5;
constexpr int kNone = -1, kOpen = -2;  // no child accepted; not decided yet
struct RowInfo {
  double z, c, s;
  float mx;
  int best, chosen, tried;
};
__device__ __forceinline__ uint64_t two(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }
__device__ __forceinline__ void store_info(uint64_t* p, const RowInfo& r) {
  store_shared(p, __builtin_bit_cast(uint64_t, r.z));
  store_shared(p + 1, __builtin_bit_cast(uint64_t, r.c));
  store_shared(p + 2, __builtin_bit_cast(uint64_t, r.s));
  store_shared(p + 3, two(__builtin_bit_cast(uint32_t, r.mx), (uint32_t)r.best));
  store_shared(p + 4, two((uint32_t)r.chosen, (uint32_t)r.tried));
}
__device__ __forceinline__ RowInfo load_info(const uint64_t* p) {
  RowInfo r;
  r.z = __builtin_bit_cast(double, load_shared(p));
  r.c = __builtin_bit_cast(double, load_shared(p + 1));
  r.s = __builtin_bit_cast(double, load_shared(p + 2));
  const uint64_t a = load_shared(p + 3), b = load_shared(p + 4);
  r.mx = __builtin_bit_cast(float, (uint32_t)a);
  r.best = (int)(a >> 32);
  r.chosen = (int)(uint32_t)b;
  r.tried = (int)(b >> 32);
  return r;
}

// A logit as the definition takes it: NaN as -inf, +inf as the largest float.
__device__ __forceinline__ float finite(float v) {
  return v > -INFINITY ? fminf(v, 3.4028234663852886e38f) : -INFINITY;
}

// 2^t for t <= 0; 0 for -inf and NaN.
__device__ __forceinline__ double exp2_below(double t) {
  t = fmax(t, -1100.0);
  const double k = __builtin_rint(t), r = t - k;
  // (ln 2)^n / n!
  double p = 4.44553827187081e-10;
  p = fma(p, r, 7.054911620801121e-09);
  p = fma(p, r, 1.0178086009239696e-07);
  p = fma(p, r, 1.3215486790144305e-06);
  p = fma(p, r, 1.5252733804059838e-05);
  p = fma(p, r, 0.00015403530393381606);
  p = fma(p, r, 0.0013333558146428441);
  p = fma(p, r, 0.009618129107628477);
  p = fma(p, r, 0.055504108664821576);
  p = fma(p, r, 0.2402265069591007);
  p = fma(p, r, 0.6931471805599453);
  p = fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)k);
}
// The weight of a logit v <= m.
__device__ __forceinline__ double weight(float v, float m, double scale) {
  return exp2_below(((double)v - (double)m) * scale);
}

// Over the wave: sums of lanes 0 .. own (the same in every run), in the last
// lane that of all.
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, two(dpp_u<CTRL, ROW_MASK>(0u, (uint32_t)u),
                                        dpp_u<CTRL, ROW_MASK>(0u, (uint32_t)(u >> 32))));
}
__device__ __forceinline__ double wave_scan_d(double v) {
  v += dpp_d<kDppShr1>(v);
  v += dpp_d<kDppShr2>(v);
  v += dpp_d<kDppShr4>(v);
  v += dpp_d<kDppShr8>(v);
  v += dpp_d<kDppBcast15, 0xA>(v);
  v += dpp_d<kDppBcast31, 0xC>(v);
  return v;
}
__device__ __forceinline__ double last_lane(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, two((uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, kWave - 1),
                                        (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), kWave - 1)));
}
__device__ __forceinline__ float wave_max(float v) { return key_value(wave_max_u32(order_key(v))); }

// Shared memory of the last workgroup of a row, and of a sequence.
struct Shared {
  int kid[MOE_TREE_MAX_ROWS];   // places of a row's children
  int tok[MOE_TREE_MAX_ROWS];   // their tokens; the path
  union {
    float val[MOE_TREE_MAX_ROWS];  // their logits, -inf for those that cannot be accepted
    int chosen[MOE_TREE_MAX_ROWS];
    double w[kRowTile];            // weights of a tile
  };
  double sum[kWavesPerBlock];
  float mx[kWavesPerBlock];
  int at[kWavesPerBlock];
  int kids, last, n, tile;
  double rest;
  RowInfo info;
};

// Over the workgroup, in every thread; barriers on both sides.
__device__ __forceinline__ float block_max(Shared& s, float v) {
  v = wave_max(v);
  if ((threadIdx.x & (kWave - 1)) == 0) s.mx[threadIdx.x >> 6] = v;
  __syncthreads();
  v = s.mx[0];
#pragma unroll
  for (int w = 1; w < kWavesPerBlock; ++w) v = fmaxf(v, s.mx[w]);
  __syncthreads();
  return v;
}
__device__ __forceinline__ int block_min(Shared& s, uint32_t v) {
  v = wave_min_u32(v);
  if ((threadIdx.x & (kWave - 1)) == 0) s.at[threadIdx.x >> 6] = (int)v;
  __syncthreads();
  uint32_t m = (uint32_t)s.at[0];
#pragma unroll
  for (int w = 1; w < kWavesPerBlock; ++w) m = min(m, (uint32_t)s.at[w]);
  __syncthreads();
  return (int)m;
}
// The sum of the threads before, and of all.
struct Scan {
  double before, all;
};
__device__ __forceinline__ Scan block_scan(Shared& s, double v) {
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x >> 6;
  const double upto = wave_scan_d(v);
  if (lane == kWave - 1) s.sum[wv] = upto;
  __syncthreads();
  Scan r{0.0, 0.0};
#pragma unroll
  for (int w = 0; w < kWavesPerBlock; ++w) {
    if (w == wv) r.before = r.all;
    r.all += s.sum[w];
  }
  // Of the lane before: a sum less the own value would not be it.
  r.before += dpp_d<0x138>(upto);
  __syncthreads();
  return r;
}

// The workgroup's row, as all threads see it.
struct Row {
  int b, i, row;  // sequence, place in it, row of the batch
  TreeRows seq;
  double scale;  // log2(e) / T
  bool greedy;
};
__device__ __forceinline__ Row find_row(const SampleArgs& a, int row) {
  KvArgs k{};
  k.offs = a.tree.offs;
  k.n_seqs = a.tree.n_seqs;
  Row r{};
  r.row = row;
  r.b = kv_sequence_of(k, row);
  if (r.b < 0) return r;
  r.seq = tree_rows(a.tree, r.b);
  r.i = row - r.seq.off;
  if (r.i >= r.seq.rows) {
    r.b = -1;
    return r;
  }
  const float t = a.temp ? a.temp[r.b] : 1.f;
  r.greedy = !(t > 0.f);
  r.scale = r.greedy ? 1.0 : 1.4426950408889634 / (double)t;
  return r;
}

// The children of row i, in order: their places and tokens.  By one wave.
__device__ __forceinline__ void list_children(const SampleArgs& a, const TreeRows& seq, int i, Shared& s) {
  const int lane = threadIdx.x & (kWave - 1);
  int n = 0;
  if (!a.tree.parents) {
    n = i + 1 < seq.rows;
    if (n && lane == 0) {
      s.kid[0] = i + 1;
      s.tok[0] = a.tokens[seq.off + i + 1];
    }
  } else {
    for (int j0 = (i + 1) & ~(kWave - 1); j0 < seq.rows && n < a.tree.max_children; j0 += kWave) {
      const int j = j0 + lane;
      const bool in = j > i && j < seq.rows;
      const int token = in ? a.tokens[seq.off + j] : 0;
      const bool is = in && a.tree.parents[seq.off + j] == i;
      const uint64_t m = __ballot(is);
      const int at = n + __popcll(m & ((1ull << lane) - 1));
      if (is && at < a.tree.max_children) {
        s.kid[at] = j;
        s.tok[at] = token;
      }
      n += __popcll(m);
    }
    n = min(n, a.tree.max_children);
  }
  if (lane == 0) s.kids = n;
}

// Counts the caller in; whether it is the last of n.  The workgroup's shared
// stores are done before, and what it loads after is what the others stored.
__device__ __forceinline__ bool last_of(unsigned* ctr, int n, Shared& s) {
  wait_stores();
  __syncthreads();
  if (threadIdx.x == 0) {
    s.last = n == 1 || arrive(ctr) == (unsigned)(n - 1);
    if (s.last && n > 1) store_shared(ctr, 0u);
  }
  __syncthreads();
  return s.last;
}

// The first column of the row's first tile whose maximum is mx.
template <typename T>
__device__ __forceinline__ int first_largest(const SampleArgs& a, int row, float mx, Shared& s) {
  uint32_t tile = ~0u;
  for (int t = threadIdx.x; t < a.tiles; t += kBlock)
    if (load_shared(a.tm + (int64_t)row * a.tiles + t) == mx) {
      tile = (uint32_t)t;
      break;
    }
  const int base = block_min(s, tile) * kRowTile;
  const T* x = (const T*)a.x + (int64_t)row * a.stride;
  uint32_t col = ~0u;
  for (int c = base + (int)threadIdx.x; c < min(base + kRowTile, a.V); c += kBlock)
    if (finite((float)x[c]) == mx) {
      col = (uint32_t)c;
      break;
    }
  return block_min(s, col);
}

// The row's sums from its tiles'.  kWithKids: and from its children, in s.val.
template <bool kWithKids>
__device__ __forceinline__ RowInfo join_row(const SampleArgs& a, const Row& r, Shared& s) {
  const float* tm = a.tm + (int64_t)r.row * a.tiles;
  const double* tz = a.tz + (int64_t)r.row * a.tiles;
  RowInfo f{0.0, 0.0, 1.0, -INFINITY, kNone, kNone, 0};
  float mx = -INFINITY;
  for (int t = threadIdx.x; t < a.tiles; t += kBlock) mx = fmaxf(mx, load_shared(tm + t));
  if (kWithKids)
    for (int k = threadIdx.x; k < s.kids; k += kBlock) mx = fmaxf(mx, s.val[k]);
  f.mx = block_max(s, mx);
  if (f.mx == -INFINITY || r.greedy) return f;
  double z = 0.0;
  for (int t = threadIdx.x; t < a.tiles; t += kBlock) {
    const float m = load_shared(tm + t);
    if (m > -INFINITY) z += load_shared(tz + t) * weight(m, f.mx, r.scale);
  }
  f.z = block_scan(s, z).all;
  return f;
}

// Drawn drafts from where they were left: f.s is the sum of what c leaves.  By
// one thread.  Stops at the first that is accepted, or rejected (then open).
template <typename T>
__device__ __forceinline__ void try_drawn(const SampleArgs& a, const Row& r, const Shared& s, RowInfo& f) {
  const T* x = (const T*)a.x + (int64_t)r.row * a.stride;
  const float* q = a.q + (int64_t)r.row * a.q_stride;
  f.chosen = kNone;
  while (f.tried < s.kids) {
    const int k = f.tried++, t = s.tok[k];
    if (t < 0 || t >= a.V) continue;
    if (r.greedy) {
      if (t == f.best) f.chosen = s.kid[k];
    } else if (f.z > 0.0) {
      const double qt = fmax((double)q[t], 0.0), u = (double)a.accept_u[r.seq.off + s.kid[k]];
      const double w = fmax(weight(finite((float)x[t]), f.mx, r.scale) / f.z - f.c * qt, 0.0);
      if (u * qt * f.s < w) {
        f.chosen = s.kid[k];
      } else {
        f.c += f.s;
        f.chosen = kOpen;
      }
    }
    if (f.chosen != kNone) return;
  }
}

// Given drafts: the first whose u times what is left is below its weight.
// By one wave.  f.z: the sum without them.
__device__ __forceinline__ void try_given(const SampleArgs& a, const Row& r, Shared& s, RowInfo& f) {
  const int lane = threadIdx.x & (kWave - 1);
  double tail = f.z;
  for (int k0 = (s.kids - 1) & ~(kWave - 1); k0 >= 0; k0 -= kWave) {
    // Lanes from the last child to the first: sums of those that come later.
    const int k = k0 + kWave - 1 - lane;
    const bool in = k < s.kids;
    const float v = in ? s.val[k] : -INFINITY;
    const double w = v > -INFINITY ? weight(v, f.mx, r.scale) : 0.0;
    const double u = in ? (double)a.accept_u[r.seq.off + s.kid[k]] : 1.0;
    const double upto = wave_scan_d(w);
    const uint64_t ok = __ballot(w > 0.0 && u * (tail + upto) < w);
    if (ok) f.chosen = s.kid[k0 + __builtin_clzll(ok)];
    tail += last_lane(upto);
  }
  if (f.z == 0.0) {  // the best of them, the lowest token of equal ones
    float m = -INFINITY;
    for (int k = 0; k < s.kids; ++k)
      if (s.val[k] > m || (s.val[k] == m && m > -INFINITY && s.tok[k] < f.best)) {
        m = s.val[k];
        f.best = s.tok[k];
      }
  }
}

// The path of a sequence, its last token and the outputs.  By the workgroup
// that is the last of the sequence.
template <typename T>
__device__ void finish(const SampleArgs& a, const Row& r, Shared& s) {
  const TreeRows& seq = r.seq;
  for (int j = threadIdx.x; j < seq.rows; j += kBlock)
    s.chosen[j] = (int)(uint32_t)load_shared(a.info + (int64_t)(seq.off + j) * kInfo + 4);
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0, at = 0;
    s.tok[0] = 0;
    for (;;) {
      const int to = s.chosen[at];
      if (to <= at || to >= seq.rows) break;
      at = to;
      s.tok[++n] = at;
    }
    s.n = n;
    s.info = load_info(a.info + (int64_t)(seq.off + at) * kInfo);
  }
  __syncthreads();
  const int n = s.n, i = s.tok[n], row = seq.off + i;
  const RowInfo f = s.info;
  int32_t* accepted = a.accepted + (int64_t)r.b * a.tree.max_rows;
  for (int j = threadIdx.x; j < a.tree.max_rows; j += kBlock) {
    if (j != n) accepted[j] = j < n ? a.tokens[seq.off + s.tok[j + 1]] : -1;
    if (a.path) a.path[(int64_t)r.b * a.tree.max_rows + j] = j <= n ? s.tok[j] : -1;
  }
  if (threadIdx.x == 0) a.n_acc[r.b] = n;
  if (a.vh)
    for (int j = threadIdx.x; j < a.hdim; j += kBlock)
      a.pending[(int64_t)r.b * a.hdim + j] = a.vh[(int64_t)row * a.hdim + j];
  __syncthreads();  // s.tok and s.chosen are done with

  int token = f.best;
  if (!r.greedy && f.mx > -INFINITY) {
    // The tile: threads take runs of tiles, in order.
    const float* tm = a.tm + (int64_t)row * a.tiles;
    const double* tz = a.tz + (int64_t)row * a.tiles;
    const bool less = a.q && f.c > 0.0;  // sums of (p - c q)+
    auto tile_sum = [&](int t) {
      const double z = load_shared(tz + t);
      if (less) return z;
      const float m = load_shared(tm + t);
      return m > -INFINITY ? z * weight(m, f.mx, r.scale) : 0.0;
    };
    const int run = (a.tiles + kBlock - 1) / kBlock, t0 = min((int)threadIdx.x * run, a.tiles);
    const int t1 = min(t0 + run, a.tiles);
    double mine = 0.0;
    for (int t = t0; t < t1; ++t) mine += tile_sum(t);
    const Scan sc = block_scan(s, mine);
    const double want = (double)a.sample_u[r.b] * sc.all;
    if (sc.all > 0.0) {
      // The first run that passes it; the last that holds anything where
      // rounding leaves none.
      const bool holds = mine > 0.0;
      int by = block_min(s, holds && sc.before + mine > want ? threadIdx.x : ~0u);
      if (by < 0) by = ~block_min(s, holds ? ~threadIdx.x : ~0u);
      if ((int)threadIdx.x == by) {
        double before = sc.before;
        int tile = t0, last = t0;
        double rest = 0.0;
        bool found = false;
        for (int t = t0; t < t1 && !found; ++t) {
          const double z = tile_sum(t);
          if (z > 0.0) {
            last = t;
            rest = want - before;
            if (before + z > want) {
              tile = t;
              found = true;
            }
          }
          before += z;
        }
        s.tile = found ? tile : last;
        s.rest = rest;
      }
      if (threadIdx.x < kWave) {
        if (!a.q) list_children(a, seq, i, s);
        else if (threadIdx.x == 0) s.kids = 0;
      }
      __syncthreads();
      const int base = s.tile * kRowTile;
      const T* x = (const T*)a.x + (int64_t)row * a.stride;
      const float* q = a.q + (int64_t)row * a.q_stride;
      for (int c = threadIdx.x; c < kRowTile; c += kBlock) {
        double w = 0.0;
        if (base + c < a.V) {
          const float v = finite((float)x[base + c]);
          if (v > -INFINITY) w = weight(v, f.mx, r.scale);
          if (less) w = fmax(w / f.z - f.c * fmax((double)q[base + c], 0.0), 0.0);
        }
        s.w[c] = w;
      }
      __syncthreads();
      for (int k = threadIdx.x; k < s.kids; k += kBlock) {
        const int c = s.tok[k] - base;
        if (s.tok[k] >= 0 && (unsigned)c < (unsigned)kRowTile) s.w[c] = 0.0;
      }
      __syncthreads();
      constexpr int kOwn = kRowTile / kBlock;
      double w[kOwn], own = 0.0;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        w[e] = s.w[threadIdx.x * kOwn + e];
        own += w[e];
      }
      double cum = block_scan(s, own).before;
      uint32_t first = ~0u, held = ~0u;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        cum += w[e];
        const uint32_t c = threadIdx.x * kOwn + e;
        if (w[e] > 0.0) {
          held = ~c;
          if (first == ~0u && cum > s.rest) first = c;
        }
      }
      int c = block_min(s, first);
      if (c < 0) c = ~block_min(s, held);
      token = base + c;
    } else if (a.q) {
      token = first_largest<T>(a, row, f.mx, s);
    }
  }
  if (threadIdx.x == 0) accepted[n] = token;
}

// Tiles' maxima and sums, each row's, and its children as far as they can be tried.
template <typename T, bool kDrawn>
__global__ __launch_bounds__(kBlock) void k_sample_rows(SampleArgs a) {
  __shared__ Shared s;
  const int lane = threadIdx.x & (kWave - 1), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int blk = blockIdx.x % a.blocks;
  const Row r = find_row(a, blockIdx.x / a.blocks);
  if (r.b < 0) return;
  constexpr int E = RowTile<T>::kElems;
  const T* x = (const T*)a.x + (int64_t)r.row * a.stride;
  const int t_end = min((blk + 1) * a.tiles_per_block, a.tiles);
  int t = blk * a.tiles_per_block + wv;
  RowTile<T> raw;
  if (t < t_end) raw.load(x, t * kRowTile, a.V, lane);
  const bool leave_out = !kDrawn && !r.greedy;
  if (leave_out) {
    if (wv == 0) list_children(a, r.seq, r.i, s);
    __syncthreads();
  }
  for (; t < t_end; t += kWavesPerBlock) {
    float v[kTileCols];
    raw.arrive();
#pragma unroll
    for (int e = 0; e < kTileCols; ++e) v[e] = finite(raw[e]);
    const int base = t * kRowTile;
    if (t + kWavesPerBlock < t_end) raw.load(x, base + kWavesPerBlock * kRowTile, a.V, lane);
    else raw.clear();
    if (leave_out)
      for (int k0 = 0; k0 < s.kids; k0 += kWave) {
        const int c = k0 + lane < s.kids ? s.tok[k0 + lane] : -1;
        for (uint64_t m = __ballot(c >= base && c < base + kRowTile); m; m &= m - 1) {
          const int at = __builtin_amdgcn_readlane(c, __builtin_ctzll(m)) - base;
          const int mine = at / (E * kWave) * E + at % E;
          if (at / E % kWave == lane)
#pragma unroll
            for (int e = 0; e < kTileCols; ++e)
              if (e == mine) v[e] = -INFINITY;
        }
      }
    float m = v[0];
#pragma unroll
    for (int e = 1; e < kTileCols; ++e) m = fmaxf(m, v[e]);
    m = wave_max(m);
    double z = 0.0;
    if (m > -INFINITY && !r.greedy) {
      double part[2] = {0.0, 0.0};
#pragma unroll
      for (int e = 0; e < kTileCols; ++e) part[e & 1] += weight(v[e], m, r.scale);
      z = wave_scan_d(part[0] + part[1]);
    }
    if (lane == kWave - 1) {
      store_shared(a.tm + (int64_t)r.row * a.tiles + t, m);
      store_shared(a.tz + (int64_t)r.row * a.tiles + t, z);
    }
  }
  if (!last_of(a.row_ctr + r.row, a.blocks, s)) return;

  if (!leave_out) {
    if (wv == 0) list_children(a, r.seq, r.i, s);
    __syncthreads();
  } else {
    // Their logits; one that an earlier child has already, or that is no
    // token, cannot be accepted.
    for (int k = threadIdx.x; k < s.kids; k += kBlock) {
      const int c = s.tok[k];
      bool ok = c >= 0 && c < a.V;
      for (int j = 0; j < k && ok; ++j) ok = s.tok[j] != c;
      s.val[k] = ok ? finite((float)x[c]) : -INFINITY;
    }
    __syncthreads();
  }
  RowInfo f;
  if (leave_out) {
    f = join_row<true>(a, r, s);
    if (f.mx > -INFINITY && wv == 0) try_given(a, r, s, f);
  } else {
    f = join_row<false>(a, r, s);
    if (f.mx > -INFINITY) {
      if (r.greedy) f.best = first_largest<T>(a, r.row, f.mx, s);
      if (threadIdx.x == 0) {
        if (kDrawn) {
          try_drawn<T>(a, r, s, f);
        } else {
          for (int k = 0; k < s.kids && f.chosen == kNone; ++k)
            if (s.tok[k] == f.best) f.chosen = s.kid[k];
        }
      }
    }
  }
  if (threadIdx.x == 0) store_info(a.info + (int64_t)r.row * kInfo, f);
  if (kDrawn) return;
  if (last_of(a.seq_ctr + r.b, r.seq.rows, s)) finish<T>(a, r, s);
}

// 16 draft probabilities of a lane, of the columns that its logits have.
template <int E>
struct ProbTile {
  float w[kTileCols];
  __device__ __forceinline__ void load(const float* row, int base, int V, int lane) {
    const float* at = row + base + lane * E;
    if (base + kRowTile <= V) {
#pragma unroll
      for (int p = 0; p < kTileCols / 4; ++p) {
        typedef float Four __attribute__((ext_vector_type(4), aligned(4)));
        const int c = (4 * p / E) * (E * kWave) + 4 * p % E;
        const Four q = __builtin_nontemporal_load(reinterpret_cast<const Four*>(at + c));
        __builtin_memcpy(w + 4 * p, &q, 16);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kTileCols; ++e) {
        const int c = (e / E) * (E * kWave) + e % E;
        w[e] = base + lane * E + c < V ? at[c] : 0.f;
      }
    }
  }
};

// Whether the path can reach the row, by what is decided so far.  Rows of this
// launch change that meanwhile, only from can to cannot: workgroups of a row
// may differ then, and what the row's sums are does not matter any more.
__device__ __forceinline__ bool reachable(const SampleArgs& a, const Row& r, Shared& s) {
  for (int j = 1 + (int)threadIdx.x; j <= r.i; j += kBlock) {
    const int p = tree_parent(a.tree, r.seq.off, j);
    bool on = false;
    if (p >= 0) {
      const int c = (int)(uint32_t)load_shared(a.info + (int64_t)(r.seq.off + p) * kInfo + 4);
      on = c == j || c == kOpen;
    }
    s.chosen[j] = on ? p : kNone;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int at = r.i;
    while (at > 0) at = s.chosen[at];
    s.n = at == 0;
  }
  __syncthreads();
  return s.n;
}

// Sums of (p - c q)+ of the rows that are open, and their next children.
template <typename T>
__global__ __launch_bounds__(kBlock) void k_sample_round(SampleArgs a) {
  __shared__ Shared s;
  const int lane = threadIdx.x & (kWave - 1), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int blk = blockIdx.x % a.blocks;
  const Row r = find_row(a, blockIdx.x / a.blocks);
  if (r.b < 0) return;
  uint64_t* info = a.info + (int64_t)r.row * kInfo;
  RowInfo f = load_info(info);  // of the launch before
  if (f.chosen == kOpen) {
    const bool on = reachable(a, r, s);
    if (on) {
      const T* x = (const T*)a.x + (int64_t)r.row * a.stride;
      const float* q = a.q + (int64_t)r.row * a.q_stride;
      const double inv = 1.0 / f.z;
      const int t_end = min((blk + 1) * a.tiles_per_block, a.tiles);
      for (int t = blk * a.tiles_per_block + wv; t < t_end; t += kWavesPerBlock) {
        RowTile<T> raw;
        ProbTile<RowTile<T>::kElems> draft;
        raw.load(x, t * kRowTile, a.V, lane);
        draft.load(q, t * kRowTile, a.V, lane);
        double part[2] = {0.0, 0.0};
#pragma unroll
        for (int e = 0; e < kTileCols; ++e) {
          const double p = weight(finite(raw[e]), f.mx, r.scale) * inv;
          part[e & 1] += fmax(p - f.c * fmax((double)draft.w[e], 0.0), 0.0);
        }
        const double z = wave_scan_d(part[0] + part[1]);
        if (lane == kWave - 1) store_shared(a.tz + (int64_t)r.row * a.tiles + t, z);
      }
    }
    if (!last_of(a.row_ctr + r.row, a.blocks, s)) return;
    if (on) {
      double sum = 0.0;
      for (int t = threadIdx.x; t < a.tiles; t += kBlock) sum += load_shared(a.tz + (int64_t)r.row * a.tiles + t);
      f.s = block_scan(s, sum).all;
      if (wv == 0) list_children(a, r.seq, r.i, s);
      __syncthreads();
      if (threadIdx.x == 0) {
        try_drawn<T>(a, r, s, f);
        store_info(info, f);
      }
    }
  } else if (blk != 0) {
    return;
  }
  if (a.last && last_of(a.seq_ctr + r.b, r.seq.rows, s)) finish<T>(a, r, s);
}

struct SamplePlan {
  int tiles, blocks, tiles_per_block;
  size_t info_bytes, z_bytes, bytes;
};

SamplePlan sample_plan(int64_t rows, int64_t vocab) {
  SamplePlan p{};
  p.tiles = (int)((vocab + kRowTile - 1) / kRowTile);
  const int64_t most = (p.tiles + kWavesPerBlock - 1) / kWavesPerBlock;
  int64_t want = kSampleSpread / (rows > 0 ? rows : 1);
  want = want < 1 ? 1 : want > most ? most : want;
  // Whole rounds of the four waves.
  p.tiles_per_block = (int)((most + want - 1) / want * kWavesPerBlock);
  p.blocks = (p.tiles + p.tiles_per_block - 1) / p.tiles_per_block;
  p.info_bytes = ((size_t)rows * kInfo * 8 + 255) & ~(size_t)255;
  p.z_bytes = (size_t)rows * p.tiles * 8;
  p.bytes = kSampleCounterBytes + p.info_bytes + p.z_bytes + (size_t)rows * p.tiles * 4;
  return p;
}

int32_t sample_check(const moe_tree* tree, int64_t vocab, bool arrays) {
  const int32_t rc = tree_check(tree, arrays);
  if (rc != MOE_OK) return rc;
  if (tree->n_rows > MOE_SAMPLE_MAX_ROWS || tree->n_seqs > MOE_SAMPLE_MAX_ROWS || vocab < 1 ||
      vocab > MOE_SAMPLE_MAX_VOCAB)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

template <typename T>
void launch_sample(SampleArgs& a, unsigned grid, hipStream_t st) {
  const dim3 g(grid), t(kBlock);
  if (!a.q) {
    hipLaunchKernelGGL((k_sample_rows<T, false>), g, t, 0, st, a);
    return;
  }
  hipLaunchKernelGGL((k_sample_rows<T, true>), g, t, 0, st, a);
  for (int k = 1; k <= a.tree.max_children; ++k) {
    a.last = k == a.tree.max_children;
    hipLaunchKernelGGL(k_sample_round<T>, g, t, 0, st, a);
  }
}

}  // namespace
}  // namespace svr

using namespace svr;

extern "C" {

int32_t moe_sample_workspace_bytes(const moe_tree* tree, int64_t vocab, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const int32_t rc = sample_check(tree, vocab, false);
  if (rc != MOE_OK) return rc;
  *bytes = sample_plan(tree->n_rows, vocab).bytes;
  return MOE_OK;
}

int32_t moe_verify_sample(const moe_tree* tree, const void* logits, int32_t dtype, int64_t vocab,
                          int64_t row_stride, const int32_t* tokens, const float* draft_probs,
                          int64_t draft_stride, const float* temperature, const float* accept_u,
                          const float* sample_u, const float* verify_h, int32_t h_dim,
                          int32_t* accepted, int32_t* path, int32_t* n_accepted, float* pending_h,
                          void* workspace, size_t workspace_bytes, void* hip_stream) {
  const int32_t rc = sample_check(tree, vocab, true);
  if (rc != MOE_OK) return rc;
  const int es = kv_elem_size(dtype);
  if (!es) return MOE_ERR_DTYPE;
  if (row_stride < vocab || (draft_probs && draft_stride < vocab) || h_dim < 0 || (!verify_h && h_dim > 0))
    return MOE_ERR_SHAPE;
  if (tree->n_rows == 0 || tree->n_seqs == 0) return MOE_OK;
  if (!logits || !tokens || !accept_u || !sample_u || !accepted || !n_accepted || !workspace)
    return MOE_ERR_NULL;
  if ((verify_h == nullptr) != (pending_h == nullptr)) return MOE_ERR_NULL;
  const SamplePlan p = sample_plan(tree->n_rows, vocab);
  if (workspace_bytes < p.bytes) return MOE_ERR_WORKSPACE;
  if ((uintptr_t)logits % es || (uintptr_t)workspace % 256 ||
      ((uintptr_t)tokens | (uintptr_t)draft_probs | (uintptr_t)temperature | (uintptr_t)accept_u |
       (uintptr_t)sample_u | (uintptr_t)verify_h | (uintptr_t)accepted | (uintptr_t)path |
       (uintptr_t)n_accepted | (uintptr_t)pending_h) % 4)
    return MOE_ERR_ARG;

  SampleArgs a{};
  a.tree = tree_args(tree);
  a.x = logits;
  a.stride = row_stride;
  a.V = (int)vocab;
  a.tiles = p.tiles;
  a.blocks = p.blocks;
  a.tiles_per_block = p.tiles_per_block;
  a.tokens = tokens;
  a.q = draft_probs;
  a.q_stride = draft_stride;
  a.temp = temperature;
  a.accept_u = accept_u;
  a.sample_u = sample_u;
  a.vh = verify_h;
  a.hdim = verify_h ? h_dim : 0;
  a.accepted = accepted;
  a.path = path;
  a.n_acc = n_accepted;
  a.pending = pending_h;
  a.row_ctr = (unsigned*)workspace;
  a.seq_ctr = a.row_ctr + MOE_SAMPLE_MAX_ROWS;
  a.info = (uint64_t*)((uint8_t*)workspace + kSampleCounterBytes);
  a.tz = (double*)((uint8_t*)a.info + p.info_bytes);
  a.tm = (float*)((uint8_t*)a.tz + p.z_bytes);
  const unsigned grid = (unsigned)tree->n_rows * (unsigned)p.blocks;
  hipStream_t st = (hipStream_t)hip_stream;
  (void)hipGetLastError();
  switch (dtype) {
    case MOE_F32: launch_sample<float>(a, grid, st); break;
    case MOE_BF16: launch_sample<bf16>(a, grid, st); break;
    default: launch_sample<_Float16>(a, grid, st); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
