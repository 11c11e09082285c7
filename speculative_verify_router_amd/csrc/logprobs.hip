// Log probabilities of given tokens, entropy and top alternatives
// (include/moe_logprobs.h) in one pass over the logits, one launch.
//
// The logits are the only large input and are read once.  A wave takes tiles
// of 1024 columns of a row, 16 a lane; a lane keeps its running maximum m and
// the sums z = sum e^(x-m), t = sum e^(x-m)(x-m), rescaled when the maximum
// grows, so that no exchange is needed before the end.
//   Alternatives: a 64-bit key orders columns by value and then by lower
// column, no two alike.  A wave holds its top_k best in order, one a lane.  A
// wave's tiles come in ascending columns, so that with top_k held a later
// column has to be larger in value: a tile whose lanes' maxima are not costs
// one comparison.  Where at least top_k lanes have such a maximum (always in
// the first tile), the top_k-th best of these is a threshold first, which all
// but few columns fail.  One or two better keys are put in their places, each
// pushing those below it a lane on (about 250 clocks each, one step waiting
// for the other); more are gathered, up to 64, and placed together by how
// many of each other and of the held ones are better (about 25 clocks each).
//   Waves, then workgroups of a row are joined the same way; the last
// workgroup to arrive at the row's counter joins them and returns the
// counter to zero.
//
// Measured at 131072 columns: 512 rows of float 45 us (5.9 TB/s: the bytes),
// of bf16 31 us (4.3 TB/s: about eight instructions a value), with five
// alternatives 50 and 45 us; 4 rows of float 6 us, with 20 alternatives 14
// (placing them and joining the workgroups); 1 row 5 us.  Loads through the
// caches, which nothing is read from twice: 51 and 40 us.  Two tiles of 16-bit
// columns in flight: the same.
#include <hip/hip_runtime.h>

#include "common.h"
#include "moe_logprobs.h"
#include "row_tile.h"

namespace svr {
namespace {

// Rows of several workgroups are rows of a small batch: kLpSpread workgroups
// a call are wanted, so a row is cut only where there are at most half as many.
constexpr int kLpSpread = 1024;
constexpr size_t kLpCounterBytes = kLpSpread / 2 * sizeof(unsigned);
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LpArgs {
  const void* x;
  int64_t stride;
  int V, blocks, tiles_per_block, k;
  const int32_t* targets;
  float *logprobs, *entropy, *top_logprobs;
  int32_t* top_ids;
  unsigned* ctr;
  uint64_t* part;  // [row]: [block][2] of (m, z), (t, 0), then [block][k] keys
};

struct Sums {
  float m, z, t;
};
// The sums of s relative to the maximum m >= s.m.
__device__ __forceinline__ Sums lp_relative(const Sums& s, float m) {
  if (s.m == m) return s;
  const float d = s.m - m, f = __builtin_amdgcn_exp2f(d * kLog2e);
  // f is 0 far below the maximum, where d may be -inf.
  return Sums{m, s.z * f, f == 0.f ? 0.f : (s.t + s.z * d) * f};
}
__device__ __forceinline__ Sums lp_join(const Sums& a, const Sums& b) {
  const float m = fmaxf(a.m, b.m);
  const Sums x = lp_relative(a, m), y = lp_relative(b, m);
  return Sums{m, x.z + y.z, x.t + y.t};
}
// Over the wave, in every lane.
__device__ __forceinline__ Sums lp_wave_join(const Sums& s) {
  const Sums x = lp_relative(s, key_value(wave_max_u32(order_key(s.m))));
  return Sums{x.m, wave_sum(x.z), wave_sum(x.t)};
}

// Columns by value, then by lower column; 0 is below every column.
__device__ __forceinline__ uint64_t lp_key(float v, uint32_t col) {
  return (uint64_t)order_key(v) << 32 | (uint32_t)~col;
}

// A bound that at least k of the wave's words v reach (there are as many): the
// upper 16 bits of the k-th largest, found two at a time, or less where
// exactly k reach it.
__device__ __forceinline__ uint32_t lp_bound(uint32_t v, int k) {
  uint32_t low = 0;
  for (int bit = 30; bit >= 16; bit -= 2) {
    int n[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) n[q] = __popcll(__ballot(v >= (low | (uint32_t)(q + 1) << bit)));
    const int q = n[2] >= k ? 3 : n[1] >= k ? 2 : n[0] >= k ? 1 : 0;
    low |= (uint32_t)q << bit;
    if (q && n[q - 1] == k) break;
  }
  return low;
}

// The k best keys that a wave has met, in order, one a lane (0: none).
struct TopKeys {
  uint64_t* buf;  // shared memory of the wave: 64 gathered keys, 64 placed ones
  int k;
  uint64_t thr;  // a key has to be above it to be held
  uint64_t key = 0;
  int held = 0, gathered = 0;

  __device__ __forceinline__ static void fence() {
    // The wave's shared-memory operations complete in order; only the
    // compiler has to keep it.
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  __device__ __forceinline__ static uint64_t of_lane(uint64_t x, int l) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), l) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, l);
  }
  __device__ __forceinline__ void follow() {
    if (held < k) return;
    const uint64_t last = of_lane(key, k - 1);
    thr = last > thr ? last : thr;
  }

  // x: the same in every lane.
  __device__ __forceinline__ void insert(uint64_t x) {
    const int lane = threadIdx.x & (kWave - 1);
    const int at = __popcll(__ballot(key > x));
    if (at >= k) return;
    constexpr int kDppWaveShr1 = 0x138;  // from the lane before
    const uint64_t before = (uint64_t)dpp_u<kDppWaveShr1>(0u, (uint32_t)(key >> 32)) << 32 |
                            dpp_u<kDppWaveShr1>(0u, (uint32_t)key);
    key = lane < at ? key : lane == at ? x : before;
    held = min(held + 1, k);
    follow();
  }

  // The gathered keys take their places.
  __device__ __forceinline__ void place() {
    const int lane = threadIdx.x & (kWave - 1);
    fence();
    const uint64_t x = lane < gathered ? buf[lane] : 0;
    int at = 0, down = 0;
    // Eight at a time: lanes behind the last hold 0, which is above nothing.
    for (int j = 0; j < gathered; j += 8)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t other = of_lane(x, j + i);
        at += other > x;
        down += other > key;
      }
    for (int j = 0; j < held; j += 8)
#pragma unroll
      for (int i = 0; i < 8; ++i) at += of_lane(key, j + i) > x;
    uint64_t* to = buf + kWave;
    if (lane < gathered && at < k) to[at] = x;
    if (lane < held && lane + down < k) to[lane + down] = key;
    fence();
    held = min(held + gathered, k);
    gathered = 0;
    key = lane < held ? to[lane] : 0;
    follow();
  }

  // N keys a lane, key_of(e), of which pass(e) says which are to be looked at:
  // each against the threshold that the one before left, or gathered.
  template <int N, typename Pass, typename Key>
  __device__ __forceinline__ void one_by_one(Pass pass, Key key_of) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (uint64_t m = __ballot(pass(e))) {
        const uint64_t x = key_of(e);
        for (; m; m &= m - 1) insert(of_lane(x, __builtin_ctzll(m)));
      }
  }
  template <int N, typename Pass, typename Key>
  __device__ __forceinline__ void together(Pass pass, Key key_of) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (uint64_t m = __ballot(pass(e))) {
        const uint64_t x = key_of(e);
        if (gathered + __popcll(m) > kWave) {
          place();
          m &= __ballot(x > thr);
        }
        if (m >> lane & 1) buf[gathered + __popcll(m & ((1ull << lane) - 1))] = x;
        gathered += __popcll(m);
      }
    if (gathered) place();
  }

  // `best`: each lane's best value (as order_key; 0: none) of what is about
  // to come.  Where k lanes or more are above the threshold, so is the k-th
  // best of them.
  __device__ __forceinline__ void raise(uint32_t best) {
    if (__popcll(__ballot(best > (uint32_t)(thr >> 32))) < k) return;
    const uint64_t low = (uint64_t)lp_bound(best, k) << 32;
    if (low > thr) thr = low - 1;
  }
};

template <typename T>
__global__ __launch_bounds__(kBlock) void k_logprobs(LpArgs a) {
  constexpr int E = RowTile<T>::kElems;
  __shared__ uint64_t s_buf[kWavesPerBlock][2 * kWave];
  __shared__ Sums s_sums[kWavesPerBlock];
  __shared__ int s_last;
  const int lane = threadIdx.x & (kWave - 1), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int row = blockIdx.x / a.blocks, blk = blockIdx.x % a.blocks;
  const T* x = (const T*)a.x + (int64_t)row * a.stride;

  // Asked for now: the last workgroup of the row needs it at its end.
  float target = 0.f;
  bool has_target = false;
  if (a.targets && threadIdx.x == 0) {
    const int t = a.targets[row];
    has_target = t >= 0 && t < a.V;
    if (has_target) target = (float)x[t];
  }
  Sums s{-INFINITY, 0.f, 0.f};
  TopKeys top{s_buf[wv], a.k, a.k ? 0ull : ~0ull};
  // (Columns stay below 2^30 + a tile of each wave.)
  const int c_begin = blk * a.tiles_per_block * kRowTile;
  const int c_end = min(c_begin + a.tiles_per_block * kRowTile, a.V);
  RowTile<T> raw;
  int base = c_begin + wv * kRowTile;
  if (base < c_end) raw.load(x, base, a.V, lane);
  for (; base < c_end; base += kWavesPerBlock * kRowTile) {
    float v[kTileCols], mx = -INFINITY;
    raw.arrive();
#pragma unroll
    for (int e = 0; e < kTileCols; ++e) {
      v[e] = raw[e];
      mx = fmaxf(mx, v[e]);
    }
    const int next = base + kWavesPerBlock * kRowTile;
    if (next < c_end) raw.load(x, next, a.V, lane);
    else raw.clear();  // nothing kept, which would be copied in every tile
    if (mx > s.m) s = lp_join(s, Sums{mx, 0.f, 0.f});
    const float m = s.m == -INFINITY ? 0.f : s.m;
    // Four chains each, then one addition to the sums of all tiles.
    float z[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < kTileCols; ++e) {
      const float d = v[e] - m;
      const float w = __builtin_amdgcn_exp2f(d * kLog2e);
      z[e & 3] += w;
      t[e & 3] = fmaf(w, fmaxf(d, -3e38f), t[e & 3]);  // a weight of zero times a finite number
    }
    s.z += (z[0] + z[1]) + (z[2] + z[3]);
    s.t += (t[0] + t[1]) + (t[2] + t[3]);
    auto column = [&](int e) { return base + (e / E) * (E * kWave) + lane * E + e % E; };
    const uint64_t in = __ballot(mx > key_value((uint32_t)(top.thr >> 32)));
    if (top.thr == 0 || in) {
      if (top.thr == 0 || __popcll(in) >= a.k) top.raise(column(0) < a.V ? order_key(mx) : 0u);
      const float above = key_value((uint32_t)(top.thr >> 32));
      if (top.held == a.k && above > -INFINITY && __popcll(in) <= 8) {
        top.one_by_one<kTileCols>([&](int e) { return v[e] >= above; },
                                [&](int e) { return lp_key(v[e], (uint32_t)column(e)); });
      } else {  // -inf and NaN too, which no comparison of values tells apart
        uint64_t key[kTileCols];
#pragma unroll
        for (int e = 0; e < kTileCols; ++e) key[e] = column(e) < a.V ? lp_key(v[e], (uint32_t)column(e)) : 0;
        top.together<kTileCols>([&](int e) { return key[e] > top.thr; }, [&](int e) { return key[e]; });
      }
    }
  }

  s = lp_wave_join(s);
  if (lane == 0) s_sums[wv] = s;
  top.fence();
  s_buf[wv][lane] = top.key;
  __syncthreads();
  uint64_t* sums = a.part + (int64_t)row * a.blocks * (2 + a.k);
  uint64_t* keys = sums + 2 * a.blocks;
  if (wv == 0) {
    for (int w = 1; w < kWavesPerBlock; ++w) s = lp_join(s, s_sums[w]);
    if (a.k) {
      uint64_t v[kWavesPerBlock - 1];
      uint32_t best = (uint32_t)(top.key >> 32);
#pragma unroll
      for (int w = 1; w < kWavesPerBlock; ++w) {
        v[w - 1] = s_buf[w][lane];
        best = max(best, (uint32_t)(v[w - 1] >> 32));
      }
      top.raise(best);
      top.together<kWavesPerBlock - 1>([&](int e) { return v[e] > top.thr; }, [&](int e) { return v[e]; });
    }
    if (a.blocks > 1) {
      if (lane == 0) {
        store_shared<uint64_t>(sums + 2 * blk, (uint64_t)__builtin_bit_cast(uint32_t, s.z) << 32 |
                                                   __builtin_bit_cast(uint32_t, s.m));
        store_shared<uint64_t>(sums + 2 * blk + 1, __builtin_bit_cast(uint32_t, s.t));
      }
      if (lane < a.k) store_shared<uint64_t>(keys + blk * a.k + lane, top.key);
      wait_stores();
    }
  }
  if (a.blocks > 1) {
    __syncthreads();
    if (threadIdx.x == 0) s_last = arrive(a.ctr + row) == (unsigned)(a.blocks - 1);
    __syncthreads();
    if (!s_last) return;
  }
  if (wv != 0) return;

  if (a.blocks > 1) {
    const int n = a.blocks * a.k;
    s = Sums{-INFINITY, 0.f, 0.f};
    top = TopKeys{s_buf[0], a.k, a.k ? 0ull : ~0ull};
    for (int b = lane; b < a.blocks; b += kWave) {
      const uint64_t mz = load_shared(sums + 2 * b), t = load_shared(sums + 2 * b + 1);
      s = lp_join(s, Sums{__builtin_bit_cast(float, (uint32_t)mz),
                          __builtin_bit_cast(float, (uint32_t)(mz >> 32)),
                          __builtin_bit_cast(float, (uint32_t)t)});
    }
    // The blocks' keys, some a lane at a time.
    constexpr int kAtOnce = 16;
    for (int i = 0; i < n; i += kAtOnce * kWave) {
      uint64_t v[kAtOnce];
      uint32_t best = 0;
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const int j = i + e * kWave + lane;
        v[e] = j < n ? load_shared(keys + j) : 0;
      }
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) best = max(best, (uint32_t)(v[e] >> 32));
      top.raise(best);
      top.together<kAtOnce>([&](int e) { return v[e] > top.thr; }, [&](int e) { return v[e]; });
    }
    s = lp_wave_join(s);
    if (lane == 0) __hip_atomic_store(a.ctr + row, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

  const bool none = s.z == 0.f;  // -inf everywhere
  const float lz = __builtin_amdgcn_logf(s.z) * kLn2;
  if (lane == 0) {
    if (a.logprobs) {
      float lp = NAN;
      if (has_target) lp = none ? -INFINITY : (target - s.m) - lz;
      a.logprobs[row] = lp;
    }
    if (a.entropy) a.entropy[row] = none ? 0.f : lz - s.t / s.z;
  }
  if (lane < a.k) {
    const int64_t at = (int64_t)row * a.k + lane;
    if (a.top_ids) a.top_ids[at] = (int32_t)~(uint32_t)top.key;
    if (a.top_logprobs)
      a.top_logprobs[at] = none ? -INFINITY : (key_value((uint32_t)(top.key >> 32)) - s.m) - lz;
  }
}

struct LpPlan {
  int blocks, tiles_per_block;
  size_t bytes;
};

// Workgroups of a row: enough for the chip when there are few rows, none
// with less than a tile a wave.
LpPlan lp_plan(int64_t rows, int64_t vocab, int k) {
  LpPlan p{};
  const int64_t tiles = (vocab + kRowTile - 1) / kRowTile;
  const int64_t most = (tiles + kWavesPerBlock - 1) / kWavesPerBlock;
  int64_t want = kLpSpread / (rows > 0 ? rows : 1);
  want = want < 1 ? 1 : want > most ? most : want;
  // Whole rounds of the four waves.
  const int64_t rounds = (most + want - 1) / want;
  p.tiles_per_block = (int)(rounds * kWavesPerBlock);
  p.blocks = (int)((tiles + p.tiles_per_block - 1) / p.tiles_per_block);
  p.bytes = kLpCounterBytes + (p.blocks > 1 ? (size_t)rows * p.blocks * (2 + k) * 8 : 0);
  return p;
}

int32_t lp_check(int32_t rows, int64_t vocab, int32_t k) {
  if (rows < 0 || rows > MOE_LOGPROBS_MAX_ROWS || vocab < 1 || vocab > MOE_LOGPROBS_MAX_VOCAB ||
      k < 0 || k > MOE_LOGPROBS_MAX_TOP || k > vocab)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

}  // namespace
}  // namespace svr

using namespace svr;

extern "C" {

int32_t moe_logprobs_workspace_bytes(int32_t max_rows, int64_t vocab, int32_t max_top,
                                     size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const int32_t rc = lp_check(max_rows, vocab, max_top);
  if (rc != MOE_OK) return rc;
  // Fewer rows are cut into more parts: the largest need of any count up to max_rows.
  size_t most = kLpCounterBytes;
  for (int64_t r = 1; r <= max_rows && r <= kLpSpread / 2; ++r) {
    const size_t n = lp_plan(r, vocab, max_top).bytes;
    most = n > most ? n : most;
  }
  *bytes = most;
  return MOE_OK;
}

int32_t moe_logprobs(const void* logits, int32_t dtype, int32_t n_rows, int64_t vocab,
                     int64_t row_stride, const int32_t* targets, float* logprobs, float* entropy,
                     int32_t top_k, int32_t* top_ids, float* top_logprobs, void* workspace,
                     size_t workspace_bytes, void* hip_stream) {
  const int32_t rc = lp_check(n_rows, vocab, top_k);
  if (rc != MOE_OK) return rc;
  const int es = dtype == MOE_F32 ? 4 : dtype == MOE_BF16 || dtype == MOE_F16 ? 2 : 0;
  if (!es) return MOE_ERR_DTYPE;
  if (row_stride < vocab) return MOE_ERR_SHAPE;
  if (n_rows == 0) return MOE_OK;
  if (!logits || !workspace || (targets == nullptr) != (logprobs == nullptr)) return MOE_ERR_NULL;
  const LpPlan p = lp_plan(n_rows, vocab, top_k);
  if (workspace_bytes < p.bytes) return MOE_ERR_WORKSPACE;
  if ((uintptr_t)logits % es || (uintptr_t)workspace % 256) return MOE_ERR_ARG;
  if (((uintptr_t)targets | (uintptr_t)logprobs | (uintptr_t)entropy | (uintptr_t)top_ids |
       (uintptr_t)top_logprobs) % 4)
    return MOE_ERR_ARG;

  LpArgs a{};
  a.x = logits;
  a.stride = row_stride;
  a.V = (int)vocab;
  a.blocks = p.blocks;
  a.tiles_per_block = p.tiles_per_block;
  a.k = top_k;
  a.targets = targets;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.ctr = (unsigned*)workspace;
  a.part = (uint64_t*)((uint8_t*)workspace + kLpCounterBytes);
  const dim3 g((unsigned)((int64_t)n_rows * p.blocks)), t(kBlock);
  hipStream_t st = (hipStream_t)hip_stream;
  (void)hipGetLastError();
  switch (dtype) {
    case MOE_F32: hipLaunchKernelGGL(k_logprobs<float>, g, t, 0, st, a); break;
    case MOE_BF16: hipLaunchKernelGGL(k_logprobs<__bf16>, g, t, 0, st, a); break;
    default: hipLaunchKernelGGL(k_logprobs<_Float16>, g, t, 0, st, a); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
