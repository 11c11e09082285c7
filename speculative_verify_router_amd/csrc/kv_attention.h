// Attention over the paged 4-bit cache (include/moe_kv.h), one kernel for
// single tokens, verify batches and prefill rows, and with masks for the rows of
// trees (include/moe_tree.h).
//
// A workgroup takes one key/value head of one sequence, 16 * RT of the rows
// that read it (row = new token x query head of the group, so four drafts of
// sixteen heads share every key that is read) and a stretch of the tokens;
// its waves take 32 tokens of the stretch in turn, each with a softmax of its
// own, joined at the end: no wave waits for another.
//   Scores are taken transposed, S^T = K Q^T, so that a lane holds four
// tokens of one row: the maximum and sum of a row need no exchange inside a
// tile, and the weights are at once the right operand of O^T = V^T P^T.
//   Keys go from memory to registers: a lane's 16 bytes are 32 channels of
// one token under one scale, four k-steps of the 16x16x32 product (the
// channels of a step are permuted, the same way in the query).  Values need
// channels as rows: they are widened, staged as [token][channel] in the
// wave's own shared memory and read back transposed.  E2M1 times a power of
// two is exact in bf16, so keys and values enter exactly.
//   Terms of bf16, of 8 bits each, hold a query value and a softmax weight: a
// query value as many as its type needs (one for bf16, two for fp16, three for
// fp32), a weight two (16 bits), three for fp32.  One term a weight would
// not do for bf16 either: the weights' roundings are independent, so they
// shrink with the number of tokens, but so does the result, and its error
// becomes as large as its own rounding (60000 tokens: 0.0023 of the result
// instead of the 0.0016 that the rounding alone makes; two terms: 0.0016).  It
// would save a third of the products (458 and 581 us for the first call below, on
// one card, when two terms took that long).
//
// Bound: instructions.  A wave alone on its SIMD issues one in about 8 clocks,
// two waves one in 4.4 together, and the registers of two row tiles leave two.
// A tile of two row tiles at D = 192 takes about 460: 96 widenings, 72 products,
// which run beside the others, 16 exponentials, 36 moves through shared memory
// and some 240 others (526 in all when every load had an address of its own and
// a weight was split alone: 8%).  Measured with 64 query on 4 key/value heads of
// 192, 512 rows over 16384 tokens: 526 us in bf16 (770 TFLOP/s, 64 to 70% of what
// a large bf16 product of the library reaches here, with a half more products
// than that counts), 846 in fp16 and 1019 in fp32 (398 TFLOP/s, three products
// each); from card to card up to a tenth more.  61 rows of a tree over 60000
// tokens 256 us (704 TFLOP/s).  4 rows over 60000 tokens 30 us with the joining
// (49 MB).  1 row: 4.5 us with one tile, 5.5 with one for each wave, 1.2 for
// every further one of a wave, and 2.9 where parts are joined: 9.5 over 777
// tokens, 20.8 over 60000 (the second kernel, and a third of the rate of the
// cache's bytes).  29 sequences of up to 5000 tokens, fp16, 32 on 8 heads of 128:
// 24 us (82 MB, 3.4 TB/s); with trees of up to 26 rows 71 (280 TFLOP/s; two products
// for one that counts, and row and token tiles that are not full make them 2.5,
// so 710 are issued where 61 rows over 60000 tokens issue 1070: 94 tiles for each
// workgroup that runs at once would be even, and the parts end at 124).
// Addresses by vector arithmetic in every tile instead of once: 892 and 1056 us
// in fp16 and fp32, 1 us for 4 rows.
// Others that were measured, for the first bf16 call, the verify batch and the
// single row, with one term a weight (458, 28.6 and 9.6 us as it was): 64 rows a
// wave (one wave a SIMD) 716 and 47 us; waves sharing widened tiles through
// shared memory, with 16x16 or 32x32 products, 475 to 497, 29 to 33 and 5.6 to
// 7.3 us (with a second kernel after the last two); eight waves in every
// workgroup 478, 33 and 11 us.
#pragma once

#include "kv.h"

namespace svr {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

// Whole division by a number that the host knows: n / d for n < 2^31 is
// n m >> s with s = 31 + ceil(log2 d), m = floor(2^s / d) + 1 (32 bits): m d
// passes 2^s by at most 2^(s - 31), which is too little to count below 2^31.
struct Divider {
  uint32_t m, s;
  int d;
  __device__ __forceinline__ int of(int n) const { return (int)((uint64_t)(uint32_t)n * m >> s); }
};
inline Divider make_divider(int d) {
  uint32_t s = 31;
  while ((int64_t)1 << (s - 31) < d) ++s;
  return Divider{(uint32_t)(((uint64_t)1 << s) / (uint64_t)d + 1), s, d};
}

struct AttnArgs {
  KvArgs kv;
  const void* q;
  int64_t qs;
  const uint8_t* cache;
  void* out;
  float* lse;
  // Parts: D sums not yet divided, and their maximum (base 2) and sum.  Where
  // the workgroup that makes the last one joins them, [part][key/value head]
  // [row of the row tile]: only row tiles that are cut have parts, so there are
  // at most two for each piece of work that runs at once, whatever the batch
  // is.  For a second kernel, [part row][head][split]; a part row is a row of
  // the batch, or row m of sequence b as b * max_rows + m where those are fewer
  // (a padded batch).
  float* part_o;
  float2* part_ml;
  unsigned* ctr;  // [row tile that is cut][key/value head] parts made, or NULL: a second kernel joins
  float c;         // scale * log2(e)
  int row_tiles, min_tiles, by_seq, search;
  int even_tiles;  // all splits are used where they have so many tiles, whatever runs at once
  int reach;  // tokens that a window's row tile lies over at most, with its first and last tile's
  // Rows of a tree (moe_tree.h): the new rows that each row sees, in 32-bit words; NULL: those before it.
  const uint32_t* mask;
  int mask_words;
  int first, extra;  // row tiles of all sequences; room for parts behind the first ones
  // Query heads a key/value head; row tiles of a sequence; splits at most;
  // Hk; work of a head that runs at once; row tiles side by side on an XCD;
  // max_rows.
  Divider G, tiles, splits, heads, share, group, rows;
};

// Waves of a workgroup, and of one that makes parts of two row tiles, where
// they are half as many to write and join (see attn_plan).
constexpr int kAttnWaves = 4, kAttnPartWaves = 8;
constexpr int kAttnTile = 32;  // tokens of a wave's step
// Up to so many parts the workgroup that makes the last one joins them: a
// second launch costs 4 us, and a workgroup reads 32 rows of sixteen parts
// (393 KB at D = 192) in about as much.
constexpr int kJoinHere = 16;
constexpr int kAttnCounters = 4096;
constexpr int kWholeRange = 1 << 28;  // a split of any number of tiles

// A sequence's rows as the kernels use them.
struct KvRows {
  int off, rows, len, place0;  // place of row 0
};
__device__ __forceinline__ KvRows kv_rows(const KvArgs& kv, int b) {
  KvRows s;
  s.off = kv.offs[b];
  const int end = kv.offs[b + 1];
  // (Wrapping only for offsets that are not ascending from 0: then no rows.)
  s.rows = s.off >= 0 && end > s.off && end <= kv.n_tokens ? end - s.off : 0;
  s.len = min(max(kv.lens[b], 0), 1 << 28);
  s.place0 = s.len - s.rows;
  s.rows = min(s.rows, kv.max_rows);
  return s;
}

// Sums, or maxima, of lanes 0 .. own.
template <bool kMax>
__device__ __forceinline__ int wave_scan(int v) {
  auto join = [&](int x) { v = kMax ? max(v, x) : v + x; };
  join(__builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));  // 1, 2, 4, 8 lanes before, in rows
  join(__builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
  join(__builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
  join(__builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
  join(__builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));  // rows 0, 2 to 1, 3
  join(__builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));  // lane 31 to the upper half
  return v;
}

// Over the sixteen lanes of a row of lanes, in each of them.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp<0xB1>(-INFINITY, v));
  v = fmaxf(v, dpp<0x4E>(-INFINITY, v));
  v = fmaxf(v, dpp<0x141>(-INFINITY, v));
  return fmaxf(v, dpp<0x140>(-INFINITY, v));
}
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp<0xB1>(0.f, v);
  v += dpp<0x4E>(0.f, v);
  v += dpp<0x141>(0.f, v);
  return v + dpp<0x140>(0.f, v);
}

// Parts that another workgroup reads in the same launch.
__device__ __forceinline__ void store_part(float* p, const f32x4v& v) {
  struct Two { uint64_t a, b; };
  const Two x = __builtin_bit_cast(Two, v);
  store_shared<uint64_t>(reinterpret_cast<uint64_t*>(p), x.a);
  store_shared<uint64_t>(reinterpret_cast<uint64_t*>(p) + 1, x.b);
}
__device__ __forceinline__ f32x4v load_part(const float* p) {
  struct { uint64_t a, b; } x{load_shared(reinterpret_cast<const uint64_t*>(p)),
                              load_shared(reinterpret_cast<const uint64_t*>(p) + 1)};
  return __builtin_bit_cast(f32x4v, x);
}

// How the tokens of a batch are cut: a split is `per` tiles, the same for
// every sequence, so that work is even whatever the lengths are.  The
// sequences' work (row tiles x tiles, a head) over what runs at once; no more
// splits than there is room for.  Whole numbers, so that the kernels agree;
// every wave finds them for itself, a lane a sequence, where there is
// something to cut.
struct KvCut {
  int row_tiles, tiles;  // of a sequence: row tiles, tiles that one of them sees at most
};
__device__ __forceinline__ KvCut kv_cut(const AttnArgs& a, const KvRows& s) {
  KvCut c;
  const int span = 16 * a.row_tiles;
  c.row_tiles = (s.rows * a.G.d + span - 1) / span;
  int seen = min(s.len, a.kv.pages_per_seq << a.kv.page_shift);
  if (a.kv.window) seen = min(seen, a.reach);
  c.tiles = (seen + kAttnTile - 1) / kAttnTile;
  return c;
}
__device__ __forceinline__ KvRows kv_lane_rows(const AttnArgs& a, int b) {
  KvRows s = kv_rows(a.kv, min(b, a.kv.n_seqs - 1));  // with no branch, so that several can be asked for at once
  if (b >= a.kv.n_seqs && a.kv.n_seqs > 1) s = KvRows{0, 0, 0, 0};  // (one sequence: in every lane)
  return s;
}
// Row tiles of all sequences in one row, with no counting: those of sequence b
// begin at floor(offs[b] G / span) + b, which leaves room for all of them (and
// for one more at most), so there are n_tokens G / span + n_seqs at most, and
// the sequence of one is found among the offsets alone, by a search that probes
// 64 at a time.  With max_rows row tiles for each sequence instead, one prompt
// of 2048 rows among 1024 single ones (200 to 3000 tokens) takes 4.8 ms, not 0.8.
__device__ __forceinline__ int kv_first_tile(const AttnArgs& a, int off, int b) {
  return (int)((uint32_t)off * (uint32_t)a.G.d >> (a.row_tiles == 2 ? 5 : 4)) + b;
}
__device__ __forceinline__ int kv_sequence_of_tile(const AttnArgs& a, int at) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, n = a.kv.n_seqs;
  while (n > 1) {
    const int step = (n + kWave - 1) / kWave, i = lane * step;
    const bool below = i < n && kv_first_tile(a, a.kv.offs[lo + i], lo + i) <= at;
    const int last = max(__popcll(__ballot(below)) - 1, 0);
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}
// Tiles of a split, and the most of a sequence.  s: the lane's sequence, of the first 64.
struct KvPer {
  int per, most;
};
__device__ __forceinline__ KvPer kv_per_most(const AttnArgs& a, const KvRows& s) {
  int64_t all = 0;
  int most = 0;
  if (a.kv.n_seqs == 1) {
    const KvCut c = kv_cut(a, s);
    all = (int64_t)c.row_tiles * c.tiles;
    most = c.tiles;
  } else {
    int64_t work = 0;
    const int lane = threadIdx.x & (kWave - 1);
    KvRows now = s;
    for (int b = 0; b < a.kv.n_seqs; b += kWave) {
      const KvRows next = kv_lane_rows(a, b + kWave + lane);
      const KvCut c = kv_cut(a, now);
      now = next;
      work += (int64_t)c.row_tiles * c.tiles;
      most = max(most, c.tiles);
    }
    most = __builtin_amdgcn_readlane(wave_scan<true>(most), kWave - 1);
    all = __builtin_amdgcn_readlane(wave_scan<false>((int)(work >> 20)), kWave - 1);
    all = (all << 20) + __builtin_amdgcn_readlane(wave_scan<false>((int)(work & 0xFFFFF)), kWave - 1);
  }
  // Rounded up, by the bits that the divider takes.
  const int shift = max(0, 34 - (int)__builtin_clzll(all | 1));
  const int64_t fair = (int64_t)(a.share.of((int)(all >> shift) + a.share.d - 1) + (shift ? 1 : 0)) << shift;
  const int even = a.splits.of(most + a.splits.d - 1);  // of the longest sequence, in all splits
  const int per = even >= a.even_tiles ? even : max(a.min_tiles, max((int)min(fair, (int64_t)kWholeRange), even));
  return KvPer{most <= 3 * a.min_tiles ? max(per, most) : per, most};  // four rounds of the waves take as long as joining
}
__device__ __forceinline__ int kv_per(const AttnArgs& a, const KvRows& s) { return kv_per_most(a, s).per; }


// Parts of a sequence's row tiles behind their first ones.  All sequences have
// fewer than a.extra: a part is at least (work of a head) / share tiles.
__device__ __forceinline__ int kv_extra(const KvCut& c, int per) { return c.row_tiles * ((c.tiles - 1) / per); }
// Those of the sequences before b.  s: the lane's sequence, of the first 64.
__device__ __forceinline__ int kv_extra_before(const AttnArgs& a, int b, int per, KvRows s) {
  int before = 0;
  for (int b0 = 0;; b0 += kWave) {
    if (b0) s = kv_lane_rows(a, b0 + (threadIdx.x & (kWave - 1)));
    const int n = kv_extra(kv_cut(a, s), per), upto = wave_scan<false>(n);
    if (b < b0 + kWave) return before + __builtin_amdgcn_readlane(upto, b - b0) - __builtin_amdgcn_readlane(n, b - b0);
    before += __builtin_amdgcn_readlane(upto, kWave - 1);
  }
}
__device__ __forceinline__ KvRows kv_rows_of_lane(const KvRows& s, int l) {
  return KvRows{__builtin_amdgcn_readlane(s.off, l), __builtin_amdgcn_readlane(s.rows, l),
                __builtin_amdgcn_readlane(s.len, l), __builtin_amdgcn_readlane(s.place0, l)};
}

// The tokens [beg, end) that rows of places [first, last] see, in tiles from
// tb on, `per` of them a split.
struct KvRange {
  int beg, end, tb, ntile, per;
  __device__ __forceinline__ bool uses(int split) const { return split == 0 || split * per < ntile; }
  __device__ __forceinline__ bool whole() const { return ntile <= per; }  // one split
};
__device__ __forceinline__ KvRange kv_range(const AttnArgs& a, int len, int first, int last, int per) {
  KvRange r;
  r.end = min(min(len, a.kv.pages_per_seq << a.kv.page_shift), last + 1);
  r.beg = a.kv.window ? max(0, first - a.kv.window + 1) : 0;
  r.tb = r.beg & ~(kAttnTile - 1);
  r.ntile = r.end > r.beg ? (r.end - r.tb + kAttnTile - 1) / kAttnTile : 0;
  r.per = per;
  return r;
}
// With rows of a tree, whichever the row tile: from the tokens that a row with
// no mark sees to the last new row.
__device__ __forceinline__ KvRange kv_tree_range(const AttnArgs& a, const KvRows& sq, int per) {
  return kv_range(a, sq.len, sq.place0 - 1, sq.place0 + sq.rows - 1, per);
}

// The new rows that a row of a tree sees.
struct TreeMask {
  const uint32_t* words;  // of the row
  int n;                  // words
  __device__ __forceinline__ uint32_t word(int w) const { return w < 0 ? ~0u : w < n ? words[w] : 0u; }
  // Bit i: new row from + i is seen; a row below 0 is a token before the new rows, from >= -32.
  __device__ __forceinline__ uint32_t bits(int from) const {
    return __builtin_amdgcn_alignbit(word((from >> 5) + 1), word(from >> 5), from & 31);
  }
  // The first place that the row sees of those before and among the new rows
  // (from place0 on, `rows` of them), where it sees the last `window`.
  __device__ __forceinline__ int first_seen(int place0, int rows, int window) const {
    auto valid = [&](int w) { return 32 * w + 32 <= rows ? words[w] : words[w] & ((1u << (rows & 31)) - 1); };
    const int used = min(n, (rows + 31) / 32);
    int marks = 0;
    for (int w = 0; w < used; ++w) marks += __popc(valid(w));
    int skip = marks - window;  // marked rows that are too far back
    if (skip < 0) return place0 + skip;
    for (int w = 0; w < used; ++w) {
      uint32_t m = valid(w);
      const int here = __popc(m);
      if (skip < here) {
        while (skip-- > 0) m &= m - 1;
        return place0 + 32 * w + __builtin_ctz(m);
      }
      skip -= here;
    }
    return place0 + rows;  // (not reached: marks > skip)
  }
};

template <int D>
__device__ __forceinline__ constexpr int step_channel(int step, int g) {
  constexpr int kFull = 4 * (D / 128);
  return step < kFull ? 128 * (step / 4) + 32 * g + 8 * (step % 4)
                      : 128 * (D / 128) + 16 * g + 8 * (step - kFull);
}

// x as a sum of NT bf16 terms (24 bits of x with three).
template <int NT>
__device__ __forceinline__ void split_terms(float x, bf16 (&t)[NT]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    t[n] = (bf16)x;
    x -= (float)t[n];
  }
}

// Two at a time: as many conversions as pairs.
template <int NT>
__device__ __forceinline__ void split_terms(float x, float y, bf16x2 (&t)[NT]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    t[n] = __builtin_convertvector((f32x2{x, y}), bf16x2);
    x -= (float)t[n].x;
    y -= (float)t[n].y;
  }
}

// Where a lane finds its part of a token l of sixteen (a run): 32 channels in
// 16 bytes of codes for each full 128 channels, 16 in 8 bytes for a last 64,
// and the aligned dword that holds their scale, with its place there.  Runs
// begin at multiples of sixteen tokens, whose scales are whole dwords, so all
// of this is the same for every tile, and a load takes no vector arithmetic.
template <int D>
struct LanePart {
  static constexpr int kParts = (D + 127) / 128;
  uint32_t code, half, scale[kParts], at[kParts];

  __device__ __forceinline__ LanePart(int l, int g) {
    code = l * (D / 2) + 16 * g;
    half = l * (D / 2) + 8 * g;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const uint32_t n = l * (D / 32) + 4 * p + (full(p) ? g : g / 2);
      scale[p] = n & ~3u;
      at[p] = 8 * (n & 3);
    }
  }
  __device__ __forceinline__ static constexpr bool full(int p) { return 64 * (2 * p + 1) < D; }
};

// A lane's codes and scales of one token for D/4 channels.  A scale is kept
// as the dword around it: of a byte the compiler keeps eight bits from tile to
// tile, and widens them where it was loaded, which would wait for the next
// tile's codes in the middle of this one.
template <int D>
struct Codes {
  static constexpr int kParts = LanePart<D>::kParts;
  uint32_t w[D / 32];
  uint32_t e[kParts];

  // codes, scales: of the run.
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, const LanePart<D>& at) {
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      if (LanePart<D>::full(p)) {
        const uint4 v = *reinterpret_cast<const uint4*>(codes + 64 * p + at.code);
        w[4 * p] = v.x;
        w[4 * p + 1] = v.y;
        w[4 * p + 2] = v.z;
        w[4 * p + 3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(codes + 64 * p + at.half);
        w[4 * p] = v.x;
        w[4 * p + 1] = v.y;
      }
      e[p] = *reinterpret_cast<const uint32_t*>(scales + at.scale[p]);
    }
  }
  // The same with the run's offsets in its page as scalars of a buffer load.
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t page, uint32_t codes, uint32_t scales,
                                       const LanePart<D>& at) {
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      if (LanePart<D>::full(p)) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(page, at.code + 64 * p, codes, 0);
        w[4 * p] = v.x;
        w[4 * p + 1] = v.y;
        w[4 * p + 2] = v.z;
        w[4 * p + 3] = v.w;
      } else {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(page, at.half + 64 * p, codes, 0);
        w[4 * p] = v.x;
        w[4 * p + 1] = v.y;
      }
      e[p] = __builtin_amdgcn_raw_buffer_load_b32(page, at.scale[p], scales, 0);
    }
  }
  // The scale of word k, in the exponent of a float.
  __device__ __forceinline__ float scale(int k, const LanePart<D>& at) const {
    return __builtin_bit_cast(float, __builtin_amdgcn_ubfe(e[k / 4], at.at[k / 4], 8) << 23);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < D / 32; ++k) w[k] = 0;
#pragma unroll
    for (int p = 0; p < kParts; ++p) e[p] = 0x7F7F7F7Fu;
  }
};

// Eight codes times s, a power of two, as bf16 (NaN where its exponent is 255).
__device__ __forceinline__ bf16x8 widen(uint32_t w, float s) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Four rows (tokens) of 16 channels, transposed: lane n of 16 gets channel n.
__device__ __forceinline__ s16x4 read_transposed(const uint8_t* p) {
  typedef __attribute__((address_space(3))) s16x4 lds4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
}

// Four sums in the output's type, aligned as one element is.
template <typename T>
__device__ __forceinline__ void store4(T* p, const f32x4v& v) {
  T x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = (T)v[e];
  __builtin_memcpy(p, x, sizeof(x));
}

// Waves of a SIMD, and so workgroups of a CU, that the registers are to leave
// room for: the queries (D/8 a term) and sums (D/4) of the row tiles decide.
constexpr int attn_waves(int D, int RT, int NT) {
  const int n = RT * (D / 8 * NT + D / 4);
  return n <= 48 ? 4 : n <= 72 ? 3 : n <= 160 ? 2 : 1;
}

// Terms of a softmax weight, for NT of a query value: never one, see above.
constexpr int attn_weight_terms(int NT) { return NT < 2 ? 2 : NT; }

// kTree: rows of a tree see the new rows that a.mask marks.  Tiles of tokens
// before the new rows are the same; the last ones, a 32nd of the tree's rows,
// take the rows' bits from memory, asked for before the next tile's codes.
template <int D, int RT, int NT, int W, typename T, bool kTree>
__global__ __launch_bounds__(W* kWave, attn_waves(D, RT, NT)) void k_kv_attention(AttnArgs a) {
  constexpr int KS = D / 32, CB = D / 16, NP = attn_weight_terms(NT);
  // The two waves of a SIMD: one that is at its products goes first, so that
  // the other's softmax fills what they leave (61 rows over 60000 tokens, bf16,
  // 311 us without, 298 with the sums' products first, 288 with the scores'
  // too).  Of two terms a query value the scores' are too many for that, of
  // three the sums' too.
  constexpr bool kScoresFirst = RT == 2 && NT == 1, kSumsFirst = RT == 2 && NT < 3;
  constexpr int kRowBytes = 2 * D + 16;            // a staged token: the pad spreads the banks
  constexpr int kStage = kAttnTile * kRowBytes;    // a wave's staged tokens
  constexpr int kJoinRow = D + 4;                  // floats of a joined row
  constexpr int kJoin = W * 16 * kJoinRow * 4;
  constexpr int kBehind = kJoin + 16 * W * 4;  // the last row's reads pass its end
  constexpr int kMem = W * kStage > kBehind ? W * kStage : kBehind;
  __shared__ __attribute__((aligned(16))) uint8_t s_mem[kMem];
  __shared__ float s_m[W][RT * 16];
  __shared__ float2 s_ml[W][16];

  const int lane = threadIdx.x & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;

  // Work of a head is a list: the row tiles of all sequences, with the first
  // part of the tokens of each, then the other parts of those that are cut:
  // sequences, their splits, the row tiles of a split.  Heads go round the
  // XCDs, and a group of row tiles, which read the same tokens, lies eight
  // workgroups apart, on one XCD, and shares its L2.
  const int G = a.G.d;
  int kvh, at;
  {
    const int v = blockIdx.x >> 3, y = a.group.of(v), u = 8 * y + (blockIdx.x & 7);
    const int n = a.heads.of(u);
    kvh = u - n * a.heads.d;
    at = n * a.group.d + v - y * a.group.d;
  }
  const bool cut = a.splits.d > 1;
  int b = 0, tile, split = 0, per = kWholeRange;
  int before = 0, apart = a.tiles.d;  // parts of the sequences before b; between those of a row tile
  KvRows sq;
  if (a.kv.n_seqs == 1) {  // as many splits of every row tile
    split = a.tiles.of(at);
    tile = at - split * a.tiles.d;
    if (split >= a.splits.d) return;
    sq = kv_rows(a.kv, 0);
    if (cut) per = kv_per(a, sq);
  } else if (at < a.first) {
    KvRows s{0, 0, 0, 0};
    if (cut) s = kv_lane_rows(a, lane);  // asked for with the sequence's own
    if (a.search) {
      b = kv_sequence_of_tile(a, at);
      sq = kv_rows(a.kv, b);
      tile = at - kv_first_tile(a, sq.off, b);
      if (tile < 0) return;  // offsets that are not ascending
    } else {
      b = a.tiles.of(at);
      tile = at - b * a.tiles.d;
      sq = kv_rows(a.kv, b);
    }
    const KvCut c = kv_cut(a, sq);
    if (cut && c.tiles > a.min_tiles) {  // others are whole, whatever `per` is
      per = kv_per(a, s);
      if (a.ctr && c.tiles > per) before = kv_extra_before(a, b, per, s);
      apart = c.row_tiles;
    }
  } else {
    at -= a.first;
    if (!cut || at >= a.extra) return;
    KvRows s = kv_lane_rows(a, lane);
    const KvPer p = kv_per_most(a, s);
    per = p.per;
    if (p.most <= per) return;  // nothing is cut
    for (;; b += kWave) {
      if (b >= a.kv.n_seqs) return;
      if (b) s = kv_lane_rows(a, b + lane);
      const KvCut c = kv_cut(a, s);
      const int n = kv_extra(c, per), upto = wave_scan<false>(n);
      const uint64_t past = __ballot(before + upto > at);
      if (!past) {
        before += __builtin_amdgcn_readlane(upto, kWave - 1);
        continue;
      }
      const int l = __builtin_ctzll(past);
      b += l;
      before += __builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(n, l);
      apart = __builtin_amdgcn_readlane(c.row_tiles, l);
      split = (at - before) / apart;
      tile = at - before - split * apart;
      ++split;
      sq = kv_rows_of_lane(s, l);
      break;
    }
  }

  const int row_total = sq.rows * G, r0 = tile * 16 * RT;
  if ((unsigned)r0 >= (unsigned)row_total) return;
  const int r_last = min(row_total, r0 + 16 * RT) - 1;
  const int first = sq.place0 + a.G.of(r0), last = sq.place0 + a.G.of(r_last);
  const KvRange rg = kTree ? kv_tree_range(a, sq, per) : kv_range(a, sq.len, first, last, per);
  if (!rg.uses(split)) return;
  // The first part is what whole ones leave at the end: those behind it in the
  // list are then all alike, and share the chip evenly whatever their order.
  // (72 sequences of 2000 tokens 36 us, 44 with the rests among them.)
  const int used = rg.whole() ? 1 : (int)((unsigned)(rg.ntile + rg.per - 1) / (unsigned)rg.per);
  const int t_begin = (split ? split - 1 : used - 1) * rg.per;
  const int t_end = min(rg.ntile, t_begin + rg.per), t_last = t_end - 1;

  // Sixteen tokens (a run) lie in one page.  A run outside [beg, end) becomes
  // one inside; what lies in a run outside of it is dropped.
  const int P = 1 << a.kv.page_shift;
  // Read through the scalar cache: as a plain load it would be a vector load
  // whose wait holds up the tile.
  const auto table = (const __attribute__((address_space(4))) int32_t*)(a.kv.table +
                                                                        (int64_t)b * a.kv.pages_per_seq);
  const int run_lo = rg.beg & ~15, run_hi = (rg.end - 1) & ~15;
  auto run = [&](int t, int u) {
    return min(max(rg.tb + min(t, t_last) * kAttnTile + 16 * u, run_lo), run_hi);
  };
  auto page_of = [&](int t, int u) { return table[run(t, u) >> a.kv.page_shift]; };
  const LanePart<D> part(l16, g);
  // Where a run lies: its page, and the offsets of its first token there.
  const uint32_t page_bytes = (uint32_t)a.kv.page_bytes, page_step = page_bytes * (uint32_t)a.kv.Hk;  // below 2^29
  const uint8_t* head = a.cache + (int64_t)kvh * page_bytes;
  struct RunAt {
    const uint8_t* page;
    uint32_t code, scale;
  };
  auto run_at = [&](int t, int u, int page) {
    page = (unsigned)page < (unsigned)a.kv.n_pages ? page : 0;
    const uint32_t i = run(t, u) & (P - 1);
    return RunAt{head + (uint64_t)(uint32_t)page * page_step, i * (D / 2),
                 P * D + i * (D / 32)};
  };
  auto load_at = [&](const RunAt& r, uint32_t code, uint32_t scale, Codes<D>& x) {
    // Two row tiles: bound by instructions, of which a buffer load takes fewer.
    // One: by latency, of which it has more (29 sequences of up to four rows,
    // fp16, 27 us instead of 25; two row tiles 263 and 256 us for 61 rows over
    // 60000 tokens).
    if constexpr (RT == 2) x.load(make_rsrc(r.page, page_bytes), code, scale, part);
    else x.load(r.page + code, r.page + scale, part);
  };
  auto load_keys = [&](const RunAt& r, Codes<D>& x) { load_at(r, r.code, r.scale, x); };
  auto load_values = [&](const RunAt& r, Codes<D>& x) {
    load_at(r, r.code + P * (D / 2), r.scale + P * (D / 32), x);
  };

  // One tile of codes is kept in flight: keys of the next tile are asked for
  // as soon as this tile's are widened, values likewise, page numbers a tile
  // before that.
  int t = t_begin + wv;
  int page[2], next_page[2];
  Codes<D> kc[2], vc[2];
  if (t < t_end) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      page[u] = page_of(t, u);
      next_page[u] = page_of(t + W, u);
    }
    const RunAt at[2] = {run_at(t, 0, page[0]), run_at(t, 1, page[1])};
#pragma unroll
    for (int u = 0; u < 2; ++u) load_keys(at[u], kc[u]);
#pragma unroll
    for (int u = 0; u < 2; ++u) load_values(at[u], vc[u]);
  }

  // The rows' queries, and the tokens that each sees: [lo, hi].
  bf16x8 qf[RT][KS][NT];
  int lo[RT], hi[RT];
  TreeMask marks[RT];  // (unused without a tree)
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = r0 + 16 * rt + l16;
    const bool on = r < row_total;
    const int m = a.G.of(min(r, row_total - 1)), h = kvh * G + min(r, row_total - 1) - m * G;
    const int place = sq.place0 + m;
    if constexpr (kTree) {
      marks[rt] = TreeMask{a.mask + (int64_t)(sq.off + m) * a.mask_words, a.mask_words};
      hi[rt] = on ? rg.end - 1 : -1;
      lo[rt] = a.kv.window ? marks[rt].first_seen(sq.place0, sq.rows, a.kv.window) : 0;
    } else {
      hi[rt] = on ? min(place, rg.end - 1) : -1;
      lo[rt] = a.kv.window ? place - a.kv.window + 1 : 0;
    }
    const T* qp = (const T*)a.q + (int64_t)(sq.off + m) * a.qs + (int64_t)h * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      T x[8];
      __builtin_memcpy(x, qp + step_channel<D>(s, g), sizeof(x));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (NT == 1) {
          qf[rt][s][0][e] = x[e];
        } else {
          bf16 t[NT];
          split_terms<NT>((float)x[e], t);
#pragma unroll
          for (int n = 0; n < NT; ++n) qf[rt][s][n][e] = t[n];
        }
      }
    }
  }
  // Tokens between these need no mask.
  const int all_hi = min(kTree ? sq.place0 - 1 : first, rg.end - 1);
  const int all_lo = a.kv.window ? (kTree ? sq.place0 + sq.rows - 1 : last) - a.kv.window + 1 : 0;

  float mx[RT], sum[RT];
  f32x4v o[RT][CB];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    mx[rt] = -INFINITY;
    sum[rt] = 0.f;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) o[rt][cb] = f32x4v{0.f, 0.f, 0.f, 0.f};
  }
  uint8_t* stage = s_mem + wv * kStage;

  for (; t < t_end; t += W) {
    const int tok0 = rg.tb + t * kAttnTile;
    bool gone[2];  // runs on a page that is not there
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      gone[u] = (unsigned)page[u] >= (unsigned)a.kv.n_pages;
      if (gone[u]) vc[u].clear();  // whatever lies there must not meet a weight of zero
    }
    if (tok0 < rg.beg || tok0 + kAttnTile > rg.end) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tk = tok0 + 16 * u + l16;
        if (tk < rg.beg || tk >= rg.end) vc[u].clear();
      }
    }
    uint32_t see[RT];  // of a tree: bit i for token tok0 + i
    if constexpr (kTree) {
      const bool among = tok0 + kAttnTile > sq.place0;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) see[rt] = among ? marks[rt].bits(tok0 - sq.place0) : ~0u;
    }
    if constexpr (kScoresFirst) __builtin_amdgcn_s_setprio(1);
    f32x4v s[RT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][u] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const bf16x8 kf = widen(kc[u].w[k], kc[u].scale(k, part));
#pragma unroll
        for (int n = NT - 1; n >= 0; --n)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[rt][k][n], s[rt][u], 0, 0, 0);
      }
    }
    if constexpr (kScoresFirst) __builtin_amdgcn_s_setprio(0);
    const RunAt next[2] = {run_at(t + W, 0, next_page[0]), run_at(t + W, 1, next_page[1])};
#pragma unroll
    for (int u = 0; u < 2; ++u) load_keys(next[u], kc[u]);

    // Values to shared memory, widened; the next ones are asked for.
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < KS; ++k)
        *reinterpret_cast<bf16x8*>(stage + (16 * u + l16) * kRowBytes + 2 * step_channel<D>(k, g)) =
            widen(vc[u].w[k], vc[u].scale(k, part));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      load_values(next[u], vc[u]);
      page[u] = next_page[u];
      next_page[u] = page_of(t + 2 * W, u);
    }

    if (gone[0] || gone[1] || tok0 + kAttnTile - 1 > all_hi || tok0 < all_lo) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tk = tok0 + 16 * u + 4 * g + i;
            bool hidden = gone[u] || tk > hi[rt] || tk < lo[rt];
            if constexpr (kTree) hidden |= !(see[rt] >> (16 * u + 4 * g + i) & 1);
            if (hidden) s[rt][u][i] = -INFINITY;
          }
    }
    // Softmax.  The maximum in use follows only where a score passes it by
    // 2^8: weights up to 2^8 lose nothing in 32 bits, and most tiles then
    // need neither an exchange between lanes nor a rescaling of the sums.
    float top[RT];
    bool grow = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float v = s[rt][0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) v = fmaxf(v, s[rt][i / 4][i % 4]);
      top[rt] = v * a.c;
      grow |= top[rt] > mx[rt] + 8.f;
    }
    if (__ballot(grow)) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float v = top[rt];
        v = fmaxf(v, __shfl_xor(v, 16, kWave));
        v = fmaxf(v, __shfl_xor(v, 32, kWave));
        v = fmaxf(v, mx[rt]);
        const float f = v == mx[rt] ? 1.f : __builtin_amdgcn_exp2f(mx[rt] - v);
        mx[rt] = v;
        sum[rt] *= f;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) o[rt][cb] *= f;
      }
    }
    bf16x8 pf[RT][NP];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float m0 = mx[rt] == -INFINITY ? 0.f : mx[rt];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        bf16x2 x[NP];
        float p[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          p[j] = __builtin_amdgcn_exp2f(fmaf(s[rt][i / 4][i % 4 + j], a.c, -m0));
          sum[rt] += p[j];
        }
        split_terms<NP>(p[0], p[1], x);
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          pf[rt][n][i] = x[n].x;
          pf[rt][n][i + 1] = x[n].y;
        }
      }
    }

    // O^T += V^T P^T.
    if constexpr (kSumsFirst) __builtin_amdgcn_s_setprio(1);
    const uint8_t* from = stage + (4 * g + l16 / 4) * kRowBytes + 8 * (l16 % 4);
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      struct { s16x4 a, b; } v{read_transposed(from + 32 * cb),
                               read_transposed(from + 16 * kRowBytes + 32 * cb)};
      const bf16x8 vf = __builtin_bit_cast(bf16x8, v);
#pragma unroll
      for (int n = NP - 1; n >= 0; --n)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          o[rt][cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[rt][n], o[rt][cb], 0, 0, 0);
    }
    if constexpr (kSumsFirst) __builtin_amdgcn_s_setprio(0);
  }

  // Where row r of the row tile has a part, and its output.
  auto out_at = [&](int r) {
    const int rm = a.G.of(r0 + r);
    return (int64_t)(sq.off + rm) * a.kv.Hq + kvh * G + r0 + r - rm * G;
  };
  auto part_at = [&](int split, int r) {
    const int part = (split ? (split - 1) * apart : a.extra) + before + tile;
    return ((int64_t)part * a.kv.Hk + kvh) * (16 * RT) + r;
  };

  // Join the waves: sums over the common maximum, a row tile at a time.
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    sum[rt] += __shfl_xor(sum[rt], 16, kWave);
    sum[rt] += __shfl_xor(sum[rt], 32, kWave);
    if (g == 0) s_m[wv][16 * rt + l16] = mx[rt];
  }
  __syncthreads();  // also: every wave is done with its staged values
  float* join = reinterpret_cast<float*>(s_mem);
  constexpr int kJoinLanes = 4 * W, kSpan = 4 * kJoinLanes, kReads = (D + kSpan - 1) / kSpan;  // of a row
  const int jr = threadIdx.x / kJoinLanes, jc = 4 * (threadIdx.x % kJoinLanes);
  auto has = [&](int j) { return D % kSpan == 0 || jc + kSpan * j < D; };
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float m = s_m[0][16 * rt + l16];
#pragma unroll
    for (int w = 1; w < W; ++w) m = fmaxf(m, s_m[w][16 * rt + l16]);
    const float f = mx[rt] == m ? 1.f : __builtin_amdgcn_exp2f(mx[rt] - m);
    if (g == 0) s_ml[wv][l16] = make_float2(m, sum[rt] * f);
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
      *reinterpret_cast<f32x4v*>(join + (wv * 16 + l16) * kJoinRow + 16 * cb + 4 * g) = o[rt][cb] * f;
    __syncthreads();
    const int r = r0 + 16 * rt + jr;
    if (r < row_total) {
      const float M = s_ml[0][jr].x;
      float L = 0.f;
      f32x4v v[kReads];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        L += s_ml[w][jr].y;
#pragma unroll
        for (int j = 0; j < kReads; ++j) {
          // (What lies behind the row is read, and dropped.)
          const f32x4v x = *reinterpret_cast<f32x4v*>(join + (w * 16 + jr) * kJoinRow + jc + kSpan * j);
          v[j] = w ? v[j] + x : x;
        }
      }
      const int64_t at = out_at(r - r0);
      if (rg.whole()) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        T* out = (T*)a.out + at * D + jc;
#pragma unroll
        for (int j = 0; j < kReads; ++j)
          if (has(j)) store4(out + kSpan * j, v[j] * inv);
        if (jc == 0 && a.lse)
          a.lse[at] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * 0.6931471805599453f;
      } else {
        int64_t pt;
        if (a.ctr) {
          pt = part_at(split, r - r0);
        } else {
          const int64_t to_seq = a.by_seq ? (int64_t)b * a.kv.max_rows - sq.off : 0;
          pt = (at + to_seq * a.kv.Hq) * a.splits.d + split;
        }
        float* part = a.part_o + pt * D + jc;
#pragma unroll
        for (int j = 0; j < kReads; ++j)
          if (has(j)) {
            if (a.ctr) store_part(part + kSpan * j, v[j]);
            else *reinterpret_cast<f32x4v*>(part + kSpan * j) = v[j];
          }
        if (jc == 0) {
          const float2 ml = make_float2(M, L);
          if (a.ctr) store_shared<uint64_t>((uint64_t*)a.part_ml + pt, __builtin_bit_cast(uint64_t, ml));
          else a.part_ml[pt] = ml;
        }
      }
    }
    if (rt + 1 < RT) __syncthreads();
  }
  if (rg.whole() || !a.ctr) return;

  // The last workgroup of the row tiles joins the parts:
  // out = sum_s w_s O_s / sum_s w_s l_s with w_s = 2^(m_s - max m).
  wait_stores();
  __syncthreads();
  bool* s_last = reinterpret_cast<bool*>(s_ml);
  unsigned* ctr = a.ctr + (before + tile) * a.kv.Hk + kvh;
  if (threadIdx.x == 0) *s_last = arrive(ctr) == (unsigned)(used - 1);
  __syncthreads();
  if (!*s_last) return;
  if (threadIdx.x == 0) store_shared(ctr, 0u);
  float* s_w = join;  // [row][part]: w_s / sum
  for (int n = threadIdx.x; n < RT * 16 * kJoinHere; n += W * kWave) {
    static_assert(kJoinHere == 16, "a row's parts are a row of lanes");
    const int row = n / kJoinHere, part = n % kJoinHere;
    float2 ml = make_float2(-INFINITY, 0.f);
    const bool on = r0 + row < row_total;
    if (on && part < used)
      ml = __builtin_bit_cast(float2, load_shared((const uint64_t*)a.part_ml + part_at(part, row)));
    const float M = row16_max(ml.x), w = ml.x == M ? 1.f : __builtin_amdgcn_exp2f(ml.x - M);
    const float L = row16_sum(w * ml.y);
    s_w[n] = L == 0.f ? 0.f : w / L;
    if (on && part == 0 && a.lse)
      a.lse[out_at(row)] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * 0.6931471805599453f;
  }
  __syncthreads();
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = 16 * rt + jr;
    if (r0 + row >= row_total) continue;
    f32x4v v[kReads];
#pragma unroll
    for (int j = 0; j < kReads; ++j) v[j] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int part = 0; part < used; ++part) {
      const float w = s_w[row * kJoinHere + part];
      const float* from = a.part_o + part_at(part, row) * D + jc;
#pragma unroll
      for (int j = 0; j < kReads; ++j)
        if (has(j)) v[j] += w * load_part(from + kSpan * j);
    }
    T* out = (T*)a.out + out_at(row) * D + jc;
#pragma unroll
    for (int j = 0; j < kReads; ++j)
      if (has(j)) store4(out + kSpan * j, v[j]);
  }
}

template <int D>
int32_t launch_kv_attention(const AttnArgs& a, int32_t dtype, int row_tiles, int waves, int grid,
                            hipStream_t st);

// Row tiles (of 16) of a workgroup of head size D and NT terms: two, for which
// a key is widened once, where they leave two waves a SIMD.  512 rows over
// 16384 tokens, two tiles and one: D = 128, fp16 466 and 555 us, fp32 632 and
// 699; D = 192, fp16 (one wave) 1158 and 892.
constexpr int attn_most_row_tiles(int D, int NT) { return attn_waves(D, 2, NT) >= 2 ? 2 : 1; }
inline int attn_terms(int32_t dtype) { return dtype == MOE_BF16 ? 1 : dtype == MOE_F16 ? 2 : 3; }
inline int attn_row_tiles(int64_t rows, int D, int32_t dtype) {
  return rows <= 16 ? 1 : attn_most_row_tiles(D, attn_terms(dtype));
}

}  // namespace svr
