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
// a power of two times a polynomial of degree nine on [-1/2, 1/2], the one
// whose largest relative error is least (8e-14) of those that are 1 at 0.
//   Given drafts: a row's children are left out of its tiles' sums and weighed
// one by one.  At the row where the path ends all of them are rejected, so the
// tiles' sums are those of what is left, with nothing subtracted; one launch.
//   Drawn drafts: sums of (p - c q)+ need the row's sum first, and after k
// rejections the sum for k - 1: a launch for each child a row can have, which
// passes over the rows that are undecided and that the path can still reach.
//
// Bound, large: a column takes about 22 instructions of 64 bits, 4.6 clocks each
// for a wave (every kind, conversions and roundings too), so 48 sequences of three
// rows in bf16 take 12 us of arithmetic beside 7.5 of bytes; 26 us a call (without
// the weights 18), and 41 with drawn drafts, whose round takes 18 to 20 us though it
// sums 16 to 27 of 141 rows (3 us of bytes, 2 of arithmetic): a row is cut by how
// many rows there are, not by how many are open, so some 240 workgroups have work,
// each wave three tiles one after another with none asked for ahead.  A table of 32
// or 128 powers takes as many instructions with its look-ups; weights of 32 bits for
// the rows and of 64 for the last ones only, two launches, would save a tenth.
//   Small: latency, 10.6 us for 4 rows of float (with a hidden state of 4096 numbers
// 12.4, of 7168 14.0: it is copied before the path's tile is looked for): the row's
// place 0.9 us, its children 0.3, logits and weights 1.4, arrival of the row 1.2,
// its sum and children 1.4, arrival of the sequence 1.0, the path 1.2, its tile 0.9,
// the column 1.8.  16.6 us with drawn drafts.  61 rows of float (32 MB, of which a
// path needs 5) 17 us.  A last
// workgroup meets its code for the first time, so what is not a loop over columns
// is kept short: with everything inlined, and four tiles a lane in a row's sum, a
// round of drawn drafts took 18 us instead of 9.  For trees of up to four rows,
// all of which the sequence's last workgroup joins at once, without arrivals of
// the rows: 11.1 us for the 4 rows, 28.4 for the 48 chains of given drafts (26.5).
#include <hip/hip_runtime.h>

#include "kv.h"
#include "moe_sample.h"
#include "row_tile.h"
#include "tree.h"

namespace svr {
namespace {

constexpr size_t kSampleCounterBytes = 2 * MOE_SAMPLE_MAX_ROWS * sizeof(unsigned);
// Workgroups of a call that are wanted, for all rows and for the rounds of drawn
// drafts, most of whose rows are done (48 chains and 9 trees of drawn drafts:
// 41.4 and 54.7 us; with 1024 44.1 and 59.7, with 8192 42.1 and 56.4: more for the
// open rows are also more that start only to leave).
constexpr int kSampleSpread = 2048, kRoundSpread = 2048;

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

// What a row's last workgroup finds, five words: one over its sum relative to
// its maximum (given drafts: the sum without them), c and S of the drafts
// rejected so far, the maximum and a token (greedy: the largest; given drafts
// with nothing else left: the best of them), the accepted child and how many
// were tried.
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

// A logit as the definition takes it: NaN and -inf as the lowest float, which
// has no weight, +inf as the largest.  (A signalling NaN is made a quiet one
// first: the median of three would give that one back.  Of a bf16 one the
// compiler would take that as done.)
constexpr float kLargest = 3.4028234663852886e38f;
__device__ __forceinline__ float finite(float v) {
  asm("" : "+v"(v));
  return __builtin_amdgcn_fmed3f(__builtin_canonicalizef(v), -kLargest, kLargest);
}
__device__ __forceinline__ bool counts(float v) { return v > -kLargest; }

// To a whole number as the instruction does it: it stops at the type's ends,
// where a conversion in C++ means nothing.
__device__ __forceinline__ int whole(double k) {
  int i;
  asm("v_cvt_i32_f64 %0, %1" : "=v"(i) : "v"(k));
  return i;
}
// 2^t for finite t <= 0, to 8e-14 of it.
__device__ __forceinline__ double exp2_below(double t) {
#pragma clang fp contract(off)
  const double k = __builtin_rint(t), r = t - k;
  double p = 9.168151968465799e-08;
  p = fma(p, r, 1.3255182694780334e-06);
  p = fma(p, r, 1.525849287352463e-05);
  p = fma(p, r, 0.00015403456037099);
  p = fma(p, r, 0.0013333547331838614);
  p = fma(p, r, 0.00961812915917161);
  p = fma(p, r, 0.05550410873970943);
  p = fma(p, r, 0.2402265069581371);
  p = fma(p, r, 0.6931471805585506);
  p = fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, whole(k));
}
// The weight of a finite logit v <= m.  (The product is rounded before its
// whole part is taken off: of a huge one, an exact product would leave a huge rest.)
__device__ __forceinline__ double weight(float v, float m, double scale) {
#pragma clang fp contract(off)
  return exp2_below(((double)v - (double)m) * scale);
}

// The same outside of the loops over columns.  What a launch does last, its last
// workgroups do alone, with instructions that come from memory as they go: as
// one function these are fewer.
__device__ __attribute__((noinline)) double weight_once(float v, float m, double scale) { return weight(v, m, scale); }

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
__device__ __forceinline__ float wave_max(float v) { return key_value(wave_max_u32(order_key(v))); }

// Shared memory of a row's workgroup.
struct Shared {
  int kid[MOE_TREE_MAX_ROWS];  // places of the row's children
  int tok[MOE_TREE_MAX_ROWS];  // their tokens
  int chosen[MOE_TREE_MAX_ROWS];
  int path[MOE_TREE_MAX_ROWS];  // the accepted rows; the rows of a round
  double sum[kWavesPerBlock];
  int at[kWavesPerBlock];
  int kids, last, n, tile;  // n: entries of path, less one
  double rest;
  RowInfo info;
};

// Over the workgroup, in every thread; barriers on both sides.
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
__device__ __forceinline__ void set_temperature(Row& r, float t) {
  r.greedy = !(t >= 1.17549435e-38f);  // (smaller ones may read as zero, here or there)
  r.scale = r.greedy ? 1.0 : 1.4426950408889634 / fmin((double)t, 1.8446744073709552e19);
}
__device__ __forceinline__ Row find_row(const SampleArgs& a, int row) {
  Row r{};
  r.row = row;
  float t = 1.f;
  if (a.tree.n_seqs < kWave) {  // every offset and temperature at once: one wait instead of three
    const int lane = threadIdx.x & (kWave - 1);
    const int off = a.tree.offs[min(lane, a.tree.n_seqs)];
    const float temp = a.temp ? a.temp[min(lane, a.tree.n_seqs - 1)] : 1.f;
    r.b = __popcll(__ballot(lane <= a.tree.n_seqs && off <= row)) - 1;
    if (r.b >= a.tree.n_seqs) r.b = -1;
    if (r.b < 0) return r;
    r.seq = tree_rows(a.tree, __builtin_amdgcn_readlane(off, r.b), __builtin_amdgcn_readlane(off, r.b + 1));
    t = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, temp), r.b));
  } else {
    KvArgs k{};
    k.offs = a.tree.offs;
    k.n_seqs = a.tree.n_seqs;
    r.b = kv_sequence_of(k, row);
    if (r.b < 0) return r;
    r.seq = tree_rows(a.tree, r.b);
    if (a.temp) t = a.temp[r.b];
  }
  r.i = row - r.seq.off;
  if ((unsigned)r.i >= (unsigned)r.seq.rows) {
    r.b = -1;
    return r;
  }
  set_temperature(r, t);
  return r;
}

// The children of row i, in order: their places and tokens.  By one wave.  The
// next 64 rows' tokens and parents may have been asked for before it was known
// where their sequence ends.
struct Next {
  int token, parent;
};
__device__ __forceinline__ Next load_next(const SampleArgs& a, int row) {
  const int j = min(row + 1 + (int)(threadIdx.x & (kWave - 1)), a.tree.n_rows - 1);
  return Next{a.tokens[j], a.tree.parents ? a.tree.parents[j] : 0};
}
__device__ __forceinline__ void list_children(const SampleArgs& a, const TreeRows& seq, int i, Shared& s, Next next) {
  const int lane = threadIdx.x & (kWave - 1);
  int n = 0;
  for (int j0 = i + 1;;) {
    const int j = j0 + lane;
    const bool is = j < seq.rows && (a.tree.parents ? next.parent == i : j == i + 1);
    const uint64_t m = __ballot(is);
    const int at = n + __popcll(m & ((1ull << lane) - 1));
    if (is && at < a.tree.max_children) {
      s.kid[at] = j;
      s.tok[at] = next.token;
    }
    n = min(n + (int)__popcll(m), a.tree.max_children);
    j0 += kWave;
    if (!a.tree.parents || j0 >= seq.rows || n == a.tree.max_children) break;
    next = load_next(a, seq.off + j0 - 1);
  }
  if (lane == 0) s.kids = n;
}

// What a child is tried with.  Asked for while the row's logits are on their
// way, by thread k for child k: the row's last workgroup needs it at once.
struct Kid {
  float val, u, q;
};
template <typename T>
__device__ __forceinline__ Kid load_kid(const SampleArgs& a, const Row& r, const Shared& s, int k) {
  Kid c{-kLargest, 1.f, 0.f};
  if (k >= s.kids) return c;
  const int t = s.tok[k];
  if (t >= 0 && t < a.V) {
    c.val = (float)((const T*)a.x)[(int64_t)r.row * a.stride + t];
    c.u = a.accept_u[r.seq.off + s.kid[k]];
    if (a.q) c.q = a.q[(int64_t)r.row * a.q_stride + t];
  }
  return c;
}

// A counter's place: 512 in a row lie in a line of 128 bytes each.  Those of one
// line are counted one after another, however different (61 rows of 32
// workgroups each: 26 us with the counters side by side, 18 so).
__device__ __forceinline__ unsigned* counter(unsigned* ctr, int i) {
  return ctr + ((i & 511) << 5 | i >> 9);
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

// Over the workgroup, in every thread; barriers on both sides.
__device__ __forceinline__ float block_max(Shared& s, float v) {
  v = wave_max(v);
  if ((threadIdx.x & (kWave - 1)) == 0) s.at[threadIdx.x >> 6] = __builtin_bit_cast(int, v);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWavesPerBlock; ++w) v = fmaxf(v, __builtin_bit_cast(float, s.at[w]));
  __syncthreads();
  return v;
}

// The row's maximum, over its tiles' and `also`, and its sum relative to that.
struct Joined {
  float m;
  double z;
};
__device__ __forceinline__ Joined join_row(const SampleArgs& a, const Row& r, float also, Shared& s) {
  const float* tm = a.tm + (int64_t)r.row * a.tiles;
  const double* tz = a.tz + (int64_t)r.row * a.tiles;
  const int first = min((int)threadIdx.x, a.tiles - 1);
  float m = load_shared(tm + first);
  double z = load_shared(tz + first);
  if ((int)threadIdx.x >= a.tiles) z = 0.0;
  float most = fmaxf(m, also);
#pragma unroll 1
  for (int t = threadIdx.x + kBlock; t < a.tiles; t += kBlock) most = fmaxf(most, load_shared(tm + t));
  Joined j{block_max(s, most), 0.0};
  if (!counts(j.m) || r.greedy) return j;
  double sum = 0.0;
#pragma unroll 1
  for (int t = threadIdx.x;;) {
    sum += z * weight_once(m, j.m, r.scale);
    t += kBlock;
    if (t >= a.tiles) break;
    m = load_shared(tm + t);
    z = load_shared(tz + t);
  }
  j.z = block_scan(s, sum).all;
  return j;
}

__device__ __forceinline__ float of_lane(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}

// Drawn drafts from where they were left: f.s is the sum of what c leaves.
// Stops at the first that is accepted, or rejected (then open).  By one wave;
// kid: of child `lane`.
template <typename T>
__device__ __forceinline__ void try_drawn(const SampleArgs& a, const Row& r, const Shared& s, Kid kid, RowInfo& f) {
  f.chosen = kNone;
#pragma unroll 1
  while (f.tried < s.kids) {
    const int k = f.tried++, t = s.tok[k];
    if (t < 0 || t >= a.V) continue;
    if (k >= kWave) kid = load_kid<T>(a, r, s, (k & ~(kWave - 1)) + (int)threadIdx.x);
    const int l = __builtin_amdgcn_readfirstlane(k & (kWave - 1));
    const double q = fmax((double)of_lane(kid.q, l), 0.0);
    const double w = fmax(weight_once(finite(of_lane(kid.val, l)), f.mx, r.scale) * f.z - f.c * q, 0.0);
    if ((double)of_lane(kid.u, l) * q * f.s < w) {
      f.chosen = s.kid[k];
    } else {
      f.c += f.s;
      f.chosen = kOpen;
    }
    return;
  }
}

// Given drafts: the first whose u times what is left is below its weight.  By
// the workgroup; kid: of child `threadIdx.x`.  One that an earlier child has
// already, or that is no token, cannot be accepted.
template <typename T>
__device__ __forceinline__ void try_given(const SampleArgs& a, const Row& r, Shared& s, Kid kid, RowInfo& f) {
  const int lane = threadIdx.x & (kWave - 1);
  auto of_child = [&](int k) {
    Kid c = s.kids > kWave ? load_kid<T>(a, r, s, k) : kid;
    bool ok = k < s.kids;
#pragma unroll 1
    for (int j = 0; j < k && ok; ++j) ok = s.tok[j] != s.tok[k];
    c.val = ok ? finite(c.val) : -kLargest;
    return c;
  };
  Kid c{-kLargest, 1.f, 0.f};
  float most = -kLargest;
  if (threadIdx.x < kWave) {
    c = of_child(lane);
    most = c.val;
#pragma unroll 1
    for (int k = lane + kWave; k < s.kids; k += kWave) most = fmaxf(most, of_child(k).val);
  }
  const Joined j = join_row(a, r, most, s);
  f.mx = j.m;
  f.z = j.z;
  if (!counts(f.mx) || threadIdx.x >= kWave) return;
  // From the last child to the first: the sum of those that come later.
  double left = f.z;
#pragma unroll 1
  for (int k = s.kids - 1, k0 = kWave * (s.kids > kWave ? s.kids : 0); k >= 0; --k) {
    if (k < k0) {  // (more than a wave's)
      k0 = k & ~(kWave - 1);
      c = of_child(k0 + lane);
    }
    const int l = __builtin_amdgcn_readfirstlane(k & (kWave - 1));
    const float v = of_lane(c.val, l);
    if (!counts(v)) continue;
    const double w = weight_once(v, f.mx, r.scale);
    left += w;
    if (w > 0.0 && (double)of_lane(c.u, l) * left < w) f.chosen = s.kid[k];
    // Nothing else left: the best of them, the lowest token of equal ones.
    if (f.z == 0.0 && v == f.mx && (f.best < 0 || s.tok[k] < f.best)) f.best = s.tok[k];
  }
}

// The path of a sequence, its last token and the outputs.  By the workgroup
// that is the last of the sequence.
template <typename T>
__device__ void finish(const SampleArgs& a, const Row& r, Shared& s) {
  const TreeRows& seq = r.seq;
  const float sample_u = a.sample_u[r.b];
  // Each thread's first row is kept: the path's last row is likely among them.
  RowInfo mine{};
#pragma unroll 1
  for (int j = threadIdx.x; j < seq.rows; j += kBlock) {
    const RowInfo f = load_info(a.info + (int64_t)(seq.off + j) * kInfo);
    s.chosen[j] = f.chosen;
    if (j < kBlock) mine = f;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0, at = 0;
    s.path[0] = 0;
    for (;;) {
      const int to = s.chosen[at];
      if (to <= at || to >= seq.rows) break;
      at = to;
      s.path[++n] = at;
    }
    s.n = n;
  }
  __syncthreads();
  const int n = s.n, i = s.path[n], row = seq.off + i;
  if ((int)threadIdx.x == (i < kBlock ? i : 0))
    s.info = i < kBlock ? mine : load_info(a.info + (int64_t)row * kInfo);
  // Threads take runs of the row's tiles, in order.
  const float* tm = a.tm + (int64_t)row * a.tiles;
  const double* tz = a.tz + (int64_t)row * a.tiles;
  const int run = (a.tiles + kBlock - 1) / kBlock, t0 = min((int)threadIdx.x * run, a.tiles);
  const int t1 = min(t0 + run, a.tiles);
  const float m0 = load_shared(tm + min(t0, a.tiles - 1));
  const double z0 = load_shared(tz + min(t0, a.tiles - 1));
  if (!a.q && threadIdx.x < kWave) list_children(a, seq, i, s, load_next(a, row));

  int32_t* accepted = a.accepted + (int64_t)r.b * a.tree.max_rows;
#pragma unroll 1
  for (int j = threadIdx.x; j < a.tree.max_rows; j += kBlock) {
    if (j != n) accepted[j] = j < n ? a.tokens[seq.off + s.path[j + 1]] : -1;
    if (a.path) a.path[(int64_t)r.b * a.tree.max_rows + j] = j <= n ? s.path[j] : -1;
  }
  if (threadIdx.x == 0) a.n_acc[r.b] = n;
  if (a.vh)
    for (int j = threadIdx.x; j < a.hdim; j += kBlock)
      a.pending[(int64_t)r.b * a.hdim + j] = a.vh[(int64_t)row * a.hdim + j];
  __syncthreads();
  const RowInfo f = s.info;
  int token = f.best;
  if (!r.greedy && counts(f.mx)) {
    const bool less = a.q && f.c > 0.0;  // sums of (p - c q)+
    auto scaled = [&](double z, float m) { return less ? z : z * weight_once(m, f.mx, r.scale); };
    const double head = t0 < t1 ? scaled(z0, m0) : 0.0;
    double own = head;
#pragma unroll 1
    for (int t = t0 + 1; t < t1; ++t) own += scaled(load_shared(tz + t), load_shared(tm + t));
    const Scan sc = block_scan(s, own);
    const double want = (double)sample_u * sc.all;
    if (sc.all > 0.0) {
      // The first run that passes it; the last that holds anything where
      // rounding leaves none.
      const bool holds = own > 0.0;
      int by = block_min(s, holds && sc.before + own > want ? threadIdx.x : ~0u);
      if (by < 0) by = ~block_min(s, holds ? ~threadIdx.x : ~0u);
      if ((int)threadIdx.x == by) {
        double before = sc.before, z = head;
        s.tile = t0;
        s.rest = want - before;
#pragma unroll 1
        for (int t = t0; !(before + z > want);) {
          before += z;
          if (++t == t1) break;
          z = scaled(load_shared(tz + t), load_shared(tm + t));
          if (z > 0.0) {
            s.tile = t;
            s.rest = want - before;
          }
        }
      }
      __syncthreads();
      // The column: four a thread, in order.
      constexpr int kOwn = kRowTile / kBlock;
      const int base = s.tile * kRowTile, c0 = base + (int)threadIdx.x * kOwn;
      const T* x = (const T*)a.x + (int64_t)row * a.stride;
      const float* q = a.q + (int64_t)row * a.q_stride;
      double w[kOwn];
      float v[kOwn], d[kOwn];
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        const int c = min(c0 + e, a.V - 1);
        v[e] = (float)x[c];
        d[e] = less ? q[c] : 0.f;
      }
      bool left_out[kOwn] = {};
      if (!a.q)
#pragma unroll 1
        for (int k = 0; k < s.kids; ++k)
#pragma unroll
          for (int e = 0; e < kOwn; ++e) left_out[e] |= s.tok[k] == c0 + e;
      own = 0.0;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        v[e] = finite(v[e]);
        w[e] = c0 + e < a.V && counts(v[e]) && !left_out[e] ? weight_once(v[e], f.mx, r.scale) : 0.0;
        if (less) w[e] = fmax(w[e] * f.z - f.c * fmax((double)d[e], 0.0), 0.0);
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
  const int row = blockIdx.x / a.blocks;
  constexpr int E = RowTile<T>::kElems;
  const T* x = (const T*)a.x + (int64_t)row * a.stride;
  const int t_end = min((blk + 1) * a.tiles_per_block, a.tiles);
  int t = blk * a.tiles_per_block + wv;
  RowTile<T> raw;
  if (t < t_end) raw.load(x, t * kRowTile, a.V, lane);  // whatever row it is: all of them have logits
  Next next{};
  if (wv == 0) next = load_next(a, row);
  const Row r = find_row(a, row);
  if (r.b < 0) return;
  const bool leave_out = !kDrawn && !r.greedy;
  if (wv == 0) list_children(a, r.seq, r.i, s, next);
  __syncthreads();
  Kid kid{};
  if (wv == 0) kid = load_kid<T>(a, r, s, lane);
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
              if (e == mine) v[e] = -kLargest;
        }
      }
    float m = v[0];
#pragma unroll
    for (int e = 1; e < kTileCols; ++e) m = fmaxf(m, v[e]);
    m = wave_max(m);
    double z = 0.0;
    if (counts(m) && !r.greedy) {
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
  if (!last_of(counter(a.row_ctr, r.row), a.blocks, s)) return;

  RowInfo f{0.0, 0.0, 1.0, -kLargest, kNone, kNone, 0};
  if (leave_out) {
    try_given<T>(a, r, s, kid, f);
  } else {
    const Joined j = join_row(a, r, -kLargest, s);
    if (counts(j.m)) {
      if (r.greedy) {
        f.best = first_largest<T>(a, r.row, j.m, s);
#pragma unroll 1
        for (int k = s.kids - 1; k >= 0; --k)
          if (s.tok[k] == f.best) f.chosen = s.kid[k];
      } else {
        f.mx = j.m;
        f.z = 1.0 / j.z;
        if (wv == 0) try_drawn<T>(a, r, s, kid, f);
      }
    }
  }
  if (threadIdx.x == 0) store_info(a.info + (int64_t)r.row * kInfo, f);
  if (kDrawn) return;
  if (last_of(counter(a.seq_ctr, r.b), r.seq.rows, s)) finish<T>(a, r, s);
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
#pragma unroll 1
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
  int at = r.i;
  while (at > 0) at = s.chosen[at];
  return at == 0;
}

// Sums of (p - c q)+ of the rows that are open, and their next children.
template <typename T>
__global__ __launch_bounds__(kBlock) void k_sample_round(SampleArgs a) {
  __shared__ Shared s;
  const int lane = threadIdx.x & (kWave - 1), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int blk = blockIdx.x % a.blocks;
  const int row = blockIdx.x / a.blocks;
  uint64_t* info = a.info + (int64_t)row * kInfo;
  RowInfo f = load_info(info);  // of the launch before (of a row of no sequence: whatever lies there)
  const Row r = find_row(a, row);
  if (r.b < 0) return;
  if (f.chosen == kOpen) {
    const T* x = (const T*)a.x + (int64_t)r.row * a.stride;
    const float* q = a.q + (int64_t)r.row * a.q_stride;
    const int t_end = min((blk + 1) * a.tiles_per_block, a.tiles);
    int t = blk * a.tiles_per_block + wv;
    RowTile<T> raw;
    ProbTile<RowTile<T>::kElems> draft;
    if (t < t_end) {
      raw.load(x, t * kRowTile, a.V, lane);
      draft.load(q, t * kRowTile, a.V, lane);
    }
    if (wv == 0) list_children(a, r.seq, r.i, s, load_next(a, row));
    const bool on = reachable(a, r, s);  // (and a barrier)
    if (on) {
      Kid kid{};
      if (wv == 0) kid = load_kid<T>(a, r, s, lane);
      const double share = f.c / f.z;
      while (t < t_end) {
        double part[2] = {0.0, 0.0};
#pragma unroll
        for (int e = 0; e < kTileCols; ++e) {
          const double w = weight(finite(raw[e]), f.mx, r.scale);
          part[e & 1] += fmax(fma(-share, (double)fmaxf(draft.w[e], 0.f), w), 0.0);
        }
        const double z = wave_scan_d(part[0] + part[1]) * f.z;
        if (lane == kWave - 1) store_shared(a.tz + (int64_t)r.row * a.tiles + t, z);
        t += kWavesPerBlock;
        if (t < t_end) {
          raw.load(x, t * kRowTile, a.V, lane);
          draft.load(q, t * kRowTile, a.V, lane);
        }
      }
      if (!last_of(counter(a.row_ctr, r.row), a.blocks, s)) return;
      double sum = 0.0;
#pragma unroll 1
      for (int k = threadIdx.x; k < a.tiles; k += kBlock) sum += load_shared(a.tz + (int64_t)r.row * a.tiles + k);
      f.s = block_scan(s, sum).all;
      if (wv == 0) {
        try_drawn<T>(a, r, s, kid, f);
        if (lane == 0) store_info(info, f);
      }
    } else if (!last_of(counter(a.row_ctr, r.row), a.blocks, s)) {
      return;
    }
  } else if (blk != 0) {
    return;
  }
  if (a.last && last_of(counter(a.seq_ctr, r.b), r.seq.rows, s)) finish<T>(a, r, s);
}

struct SamplePlan {
  int tiles;
  size_t info_bytes, z_bytes, bytes;
};

// Workgroups of a row, and the tiles of each: whole rounds of the four waves.
void sample_cut(int64_t rows, int tiles, int64_t spread, int* blocks, int* tiles_per_block) {
  const int64_t most = (tiles + kWavesPerBlock - 1) / kWavesPerBlock;
  int64_t want = spread / (rows > 0 ? rows : 1);
  want = want < 1 ? 1 : want > most ? most : want;
  *tiles_per_block = (int)((most + want - 1) / want * kWavesPerBlock);
  *blocks = (tiles + *tiles_per_block - 1) / *tiles_per_block;
}

SamplePlan sample_plan(int64_t rows, int64_t vocab) {
  SamplePlan p{};
  p.tiles = (int)((vocab + kRowTile - 1) / kRowTile);
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
void launch_sample(SampleArgs& a, hipStream_t st) {
  const dim3 t(kBlock);
  sample_cut(a.tree.n_rows, a.tiles, kSampleSpread, &a.blocks, &a.tiles_per_block);
  const dim3 g((unsigned)a.tree.n_rows * (unsigned)a.blocks);
  if (!a.q) {
    hipLaunchKernelGGL((k_sample_rows<T, false>), g, t, 0, st, a);
    return;
  }
  hipLaunchKernelGGL((k_sample_rows<T, true>), g, t, 0, st, a);
  sample_cut(a.tree.n_rows, a.tiles, kRoundSpread, &a.blocks, &a.tiles_per_block);
  const dim3 rounds((unsigned)a.tree.n_rows * (unsigned)a.blocks);
  for (int k = 1; k <= a.tree.max_children; ++k) {
    a.last = k == a.tree.max_children;
    hipLaunchKernelGGL(k_sample_round<T>, rounds, t, 0, st, a);
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
  hipStream_t st = (hipStream_t)hip_stream;
  (void)hipGetLastError();
  switch (dtype) {
    case MOE_F32: launch_sample<float>(a, st); break;
    case MOE_BF16: launch_sample<bf16>(a, st); break;
    default: launch_sample<_Float16>(a, st); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
