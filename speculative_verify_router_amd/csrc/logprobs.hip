// Log probabilities of given tokens, entropy and top alternatives
// (include/moe_logprobs.h) in one pass over the logits, one launch.
//
// The logits are the only large input and are read once.  A wave takes tiles
// of 1024 columns of a row, 16 a lane; a lane keeps its running maximum m and
// the sums z = sum e^(x-m), t = sum e^(x-m)(x-m), rescaled when the maximum
// grows, so that no exchange is needed before the end.
//   Alternatives: a 64-bit key orders columns by value and then by lower
// column, no two alike.  A wave keeps the keys above its threshold in a short
// list in shared memory; when the list is full, it is cut to the top_k best
// and the threshold follows.  Whole tiles below the threshold cost one
// comparison of the lane's maximum, so that of 131072 random columns only a
// few hundred are ever listed.
//   Waves, then workgroups of a row are joined the same way; the last
// workgroup to arrive at the row's counter joins them and returns the
// counter to zero.
#include <hip/hip_runtime.h>

#include "common.h"
#include "moe_logprobs.h"

namespace svr {
namespace {

constexpr int kLpCols = 16;                // columns of a lane in a tile
constexpr int kLpTile = kLpCols * kWave;   // columns of a wave's tile
constexpr int kLpList = 256;               // keys a wave lists
// Rows of several workgroups are rows of a small batch: kLpSpread workgroups
// a call are wanted, so a row is cut only where there are at most half as many.
constexpr int kLpSpread = 1024;
constexpr size_t kLpCounterBytes = kLpSpread / 2 * sizeof(unsigned);
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LpArgs {
  const void* x;
  int64_t stride, V;
  int N, blocks, tiles_per_block, k, vec;
  const int32_t* targets;
  float *logprobs, *entropy, *top_logprobs;
  int32_t* top_ids;
  unsigned* ctr;
  uint64_t* part;  // [row][block][2 + k]: (m, z), (t, 0), keys
};

struct Sums {
  float m, z, t;
};
__device__ __forceinline__ Sums lp_join(const Sums& a, const Sums& b) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  // A side at the joint maximum keeps its sums (also where both are -inf).
  const float da = a.m == r.m ? 0.f : a.m - r.m, db = b.m == r.m ? 0.f : b.m - r.m;
  const float fa = __builtin_amdgcn_exp2f(da * kLog2e), fb = __builtin_amdgcn_exp2f(db * kLog2e);
  r.z = a.z * fa + b.z * fb;
  r.t = (a.z == 0.f ? 0.f : (a.t + a.z * da) * fa) + (b.z == 0.f ? 0.f : (b.t + b.z * db) * fb);
  // fa is 0 far below the maximum, where da may be -inf.
  if (fa == 0.f) r.t = b.t;
  if (fb == 0.f) r.t = a.t;
  return r;
}
__device__ __forceinline__ Sums lp_wave_join(Sums s) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    Sums b;
    b.m = __shfl_xor(s.m, o, kWave);
    b.z = __shfl_xor(s.z, o, kWave);
    b.t = __shfl_xor(s.t, o, kWave);
    s = lp_join(s, b);
  }
  return s;
}

// Columns by value, then by lower column; 0 is below every column.
__device__ __forceinline__ uint64_t lp_key(float v, uint32_t col) {
  return (uint64_t)order_key(v) << 32 | (uint32_t)~col;
}

// A wave's list of keys above a threshold.
struct TopList {
  uint64_t* buf;  // kLpList keys in shared memory
  int n, k;
  uint64_t thr;   // a key has to be above it to matter

  __device__ __forceinline__ void fence() {
    // The wave's shared-memory operations complete in order; only the
    // compiler has to keep it.
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }

  // Cut to the k largest (n >= k): bisects the key of the k-th by its bits,
  // until a bound has exactly k keys at or above it.
  __device__ void cut() {
    const int lane = threadIdx.x & (kWave - 1);
    fence();
    uint64_t v[kLpList / kWave];
#pragma unroll
    for (int j = 0; j < kLpList / kWave; ++j) v[j] = kWave * j + lane < n ? buf[kWave * j + lane] : 0;
    uint64_t lowest = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t c = lowest | 1ull << bit;
      int have = 0;
#pragma unroll
      for (int j = 0; j < kLpList / kWave; ++j) have += __popcll(__ballot(v[j] >= c));
      if (have >= k) lowest = c;
      if (have == k) break;
    }
    fence();
    int at = 0;
#pragma unroll
    for (int j = 0; j < kLpList / kWave; ++j) {
      const uint64_t keep = __ballot(v[j] >= lowest);
      if (v[j] >= lowest) buf[at + __popcll(keep & ((1ull << lane) - 1))] = v[j];
      at += __popcll(keep);
    }
    fence();
    n = at;
    thr = lowest - 1;
  }

  // Each lane offers one key (0: none).
  __device__ __forceinline__ void offer(uint64_t key) {
    uint64_t in = __ballot(key > thr);
    if (!in) return;
    if (n + __popcll(in) > kLpList) {
      cut();
      in = __ballot(key > thr);
    }
    const int lane = threadIdx.x & (kWave - 1);
    if (key > thr) buf[n + __popcll(in & ((1ull << lane) - 1))] = key;
    n += __popcll(in);
  }
};

template <typename T>
struct Piece {
  static constexpr int kElems = 16 / sizeof(T);
  static constexpr int kCount = kLpCols / kElems;
};

// 16 columns of a lane from tile column `base`: pieces of 16 bytes, lane
// after lane.  Columns from V on are -inf.
template <typename T>
__device__ __forceinline__ void lp_load(const T* row, int64_t base, int64_t V, bool vec, int lane,
                                        T (&x)[kLpCols]) {
  constexpr int E = Piece<T>::kElems;
#pragma unroll
  for (int p = 0; p < Piece<T>::kCount; ++p) {
    const int64_t c = base + p * (E * kWave) + lane * E;
    if (vec && c + E <= V) {
      *reinterpret_cast<uint4*>(x + p * E) = *reinterpret_cast<const uint4*>(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[p * E + e] = c + e < V ? row[c + e] : (T)-INFINITY;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kBlock) void k_logprobs(LpArgs a) {
  constexpr int E = Piece<T>::kElems;
  __shared__ uint64_t s_list[kWavesPerBlock][kLpList];
  __shared__ Sums s_sums[kWavesPerBlock];
  __shared__ int s_n[kWavesPerBlock], s_last;
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x >> 6;
  const int row = blockIdx.x / a.blocks, blk = blockIdx.x % a.blocks;
  const T* x = (const T*)a.x + (int64_t)row * a.stride;

  Sums s{-INFINITY, 0.f, 0.f};
  TopList top{s_list[wv], 0, a.k, a.k ? 0ull : ~0ull};
  const int64_t c_begin = (int64_t)blk * a.tiles_per_block * kLpTile;
  const int64_t c_end = min(c_begin + (int64_t)a.tiles_per_block * kLpTile, a.V);
  for (int64_t base = c_begin + wv * kLpTile; base < c_end; base += kWavesPerBlock * kLpTile) {
    T raw[kLpCols];
    lp_load(x, base, a.V, a.vec, lane, raw);
    float v[kLpCols], mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < kLpCols; ++e) {
      v[e] = (float)raw[e];
      mx = fmaxf(mx, v[e]);
    }
    if (mx > s.m) s = lp_join(s, Sums{mx, 0.f, 0.f});
    const float m = s.m == -INFINITY ? 0.f : s.m;
#pragma unroll
    for (int e = 0; e < kLpCols; ++e) {
      const float d = v[e] - m;
      const float w = __builtin_amdgcn_exp2f(d * kLog2e);
      s.z += w;
      s.t = fmaf(w, fmaxf(d, -3e38f), s.t);  // a weight of zero times a finite number
    }
    if (__ballot(order_key(mx) >= (uint32_t)(top.thr >> 32))) {
#pragma unroll
      for (int e = 0; e < kLpCols; ++e) {
        const int64_t c = base + (e / E) * (E * kWave) + lane * E + e % E;
        top.offer(c < a.V ? lp_key(v[e], (uint32_t)c) : 0ull);
      }
    }
  }

  s = lp_wave_join(s);
  if (top.n > a.k) top.cut();
  if (lane == 0) {
    s_sums[wv] = s;
    s_n[wv] = top.n;
  }
  __syncthreads();
  const int stride = 2 + a.k;
  if (wv == 0) {
    for (int w = 1; w < kWavesPerBlock; ++w) {
      s = lp_join(s, s_sums[w]);
      top.offer(lane < s_n[w] ? s_list[w][lane] : 0ull);
    }
    if (top.n > a.k) top.cut();
    top.fence();
    if (a.blocks > 1) {
      uint64_t* p = a.part + ((int64_t)row * a.blocks + blk) * stride;
      if (lane == 0) {
        store_shared<uint64_t>(p, (uint64_t)__builtin_bit_cast(uint32_t, s.z) << 32 |
                                      __builtin_bit_cast(uint32_t, s.m));
        store_shared<uint64_t>(p + 1, __builtin_bit_cast(uint32_t, s.t));
      }
      if (lane < a.k) store_shared<uint64_t>(p + 2 + lane, lane < top.n ? top.buf[lane] : 0);
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
    s = Sums{-INFINITY, 0.f, 0.f};
    top.n = 0;
    top.thr = a.k ? 0ull : ~0ull;
    const uint64_t* p = a.part + (int64_t)row * a.blocks * stride;
    for (int b = lane; b < a.blocks; b += kWave) {
      const uint64_t mz = load_shared(p + (int64_t)b * stride);
      const uint64_t t = load_shared(p + (int64_t)b * stride + 1);
      s = lp_join(s, Sums{__builtin_bit_cast(float, (uint32_t)mz),
                          __builtin_bit_cast(float, (uint32_t)(mz >> 32)),
                          __builtin_bit_cast(float, (uint32_t)t)});
    }
    s = lp_wave_join(s);
    const int keys = a.blocks * a.k;
    for (int i = 0; i < keys; i += kWave) {
      const int j = i + lane;
      top.offer(j < keys ? load_shared(p + (int64_t)(j / a.k) * stride + 2 + j % a.k) : 0ull);
    }
    if (top.n > a.k) top.cut();
    top.fence();
    if (lane == 0) __hip_atomic_store(a.ctr + row, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

  const bool none = s.z == 0.f;  // -inf everywhere
  const float lz = __builtin_amdgcn_logf(s.z) * kLn2;
  if (lane == 0) {
    if (a.logprobs) {
      const int t = a.targets[row];
      float lp = NAN;
      if (t >= 0 && t < a.V) lp = none ? -INFINITY : ((float)x[t] - s.m) - lz;
      a.logprobs[row] = lp;
    }
    if (a.entropy) a.entropy[row] = none ? 0.f : lz - s.t / s.z;
  }
  if (lane < a.k) {
    const uint64_t key = top.buf[lane];
    int rank = 0;
    for (int j = 0; j < a.k; ++j) rank += top.buf[j] > key;
    const uint32_t c = ~(uint32_t)key;
    const int64_t at = (int64_t)row * a.k + rank;
    if (a.top_ids) a.top_ids[at] = (int32_t)c;
    if (a.top_logprobs)
      a.top_logprobs[at] = none ? -INFINITY : ((float)x[c] - s.m) - lz;
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
  const int64_t tiles = (vocab + kLpTile - 1) / kLpTile;
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
  a.V = vocab;
  a.N = n_rows;
  a.blocks = p.blocks;
  a.tiles_per_block = p.tiles_per_block;
  a.k = top_k;
  a.vec = (uintptr_t)logits % 16 == 0 && row_stride * es % 16 == 0;
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
