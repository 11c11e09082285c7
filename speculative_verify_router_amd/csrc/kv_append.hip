// Head norms, position rotation and append to the paged 4-bit cache, and
// reading rows back (include/moe_kv.h).
//
// A unit is one head vector: a query head, or a key head with its value head
// (together, so that a NaN or infinity in either marks the token).  A group
// of lanes takes a unit: eight channels a lane of a query (16 bytes of a
// 16-bit type), four of a key, whose 64-bit arithmetic then fits in few
// registers and is spread over a token's waves evenly; a 4-bit block of 32
// channels is eight of its lanes, and two lanes' codes are a dword.  The pair
// of a rotated channel is in the same lane (neighbours), or is read from
// memory once more, which the cache answers.
//
// The pass is to be bound by its bytes: each of q, k, v is read once, q_out
// and the codes written once.  A workgroup serves one token: the angles
// (64-bit: at place 60000 a 32-bit angle is off by 2^-9) and the norms'
// weights go into tables of factors in shared memory, once for all its heads,
// which leaves a query's channel two products, a sum and its share of the
// norm; the first heads and the weights are asked for before anything else.
// Queries are normed and rotated in 32 bits, keys in 64, because a code is a
// whole number and a key next to a rounding border must fall on its own side
// whatever the order of the sum.
//
// q_out goes past the caches: what reads it next runs on all dies, of which
// one wrote a row, and a prefill's does not stay; through them, 1878 tokens
// take 31 us and not 25, and a call with the attention behind it the same.
//
// Measured with 64 query and 4 key/value heads of 192 channels: 1878 tokens in
// bf16 (98 MB) 25 us (3.9 TB/s; 20 without norms and rotation), 512 tokens in
// float (52 MB) 14 us; 4 tokens 4.3 us, of which the reads one after another
// (offsets, page, heads) are most.  Angles taken anew for every head: 91, 34
// and 8 us; factors in registers and one step ahead, whose copies waited for
// the stores: 50 and 26; eight channels of a key a lane: 127 registers instead
// of 81, 4.9 us for 4 tokens; two workgroups a token: 38 us.
#include <type_traits>

#include "kv.h"

namespace svr {
namespace {

struct AppendArgs {
  KvArgs kv;
  const void *q, *k, *v;
  int64_t qs, ks, vs;
  const float *q_norm, *k_norm, *inv_freq;
  const int32_t* positions;
  uint8_t* cache;
  void* q_out;
  float eps;
  int rotary, interleaved;
  int parts, k_steps, steps, steps_per_part;  // workgroups of a token; waves' steps, keys first
};

// Lanes of a query head, eight channels each, and of a key/value head, four.
constexpr int query_lanes(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }
constexpr int key_lanes(int D) { return 2 * query_lanes(D); }

// Sum over the LG lanes of a unit, in each of them.
template <int LG>
__device__ __forceinline__ float group_sum(float v) {
  v += dpp<0xB1>(0.f, v);   // lanes xor 1
  v += dpp<0x4E>(0.f, v);   // xor 2
  v += dpp<0x141>(0.f, v);  // the other four of eight
  if (LG >= 16) v += dpp<0x140>(0.f, v);  // the other eight of sixteen
  // The other sixteen of thirty-two.
  if (LG >= 32) v += __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401F));
  return v;
}
template <int CTRL>
__device__ __forceinline__ double dpp_double(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp_u<CTRL>(0u, (uint32_t)(u >> 32)) << 32 | dpp_u<CTRL>(0u, (uint32_t)u));
}
template <int LG>
__device__ __forceinline__ double group_sum(double v) {
  v += dpp_double<0xB1>(v);
  v += dpp_double<0x4E>(v);
  v += dpp_double<0x141>(v);
  v += dpp_double<0x140>(v);
#pragma unroll
  for (int m = 16; m < LG; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// Norm and rotation of a channel x: r (x A + y B), r the norm's factor, y the
// channel that x is turned with, A = w cos and B = -+ w' sin with the norm
// weights w of x and w' of y.  A and B are the same for every head of a token,
// so its workgroup puts them into shared memory first.
template <int D>
struct Tables {
  double ka[D], kb[D];
  float qa[D], qb[D];
};
// Pair j of a token's channels; those that are not turned have A = w, B = 0.
struct Pair {
  int c1, c2;
  float k1, k2, q1, q2, freq;

  __device__ __forceinline__ Pair(const AppendArgs& a, int j) {
    const int half = a.rotary / 2;
    const bool turned = j < half;
    c1 = turned && !a.interleaved ? j : 2 * j;
    c2 = turned && !a.interleaved ? j + half : 2 * j + 1;
    k1 = k2 = q1 = q2 = 1.f;
    if (a.k_norm) k1 = a.k_norm[c1], k2 = a.k_norm[c2];
    if (a.q_norm) q1 = a.q_norm[c1], q2 = a.q_norm[c2];
    freq = turned ? a.inv_freq[j] : 0.f;
  }
  template <int D>
  __device__ __forceinline__ void fill(Tables<D>& t, double pos, bool keys, bool queries) const {
    double sn = 0.0, cn = 1.0;
    if (freq != 0.f) sincos(pos * (double)freq, &sn, &cn);
    if (keys) {
      t.ka[c1] = k1 * cn;
      t.ka[c2] = k2 * cn;
      t.kb[c1] = -(k2 * sn);
      t.kb[c2] = k1 * sn;
    }
    if (queries) {
      t.qa[c1] = (float)(q1 * cn);
      t.qa[c2] = (float)(q2 * cn);
      t.qb[c1] = (float)-(q2 * sn);
      t.qb[c2] = (float)(q1 * sn);
    }
  }
};
__device__ __forceinline__ float norm_factor(float mean) {
  // The instruction (1 ulp) takes subnormal numbers for zeros.
  const bool tiny = mean < 1e-30f;
  const float r = __builtin_amdgcn_rsqf(tiny ? mean * 0x1p100f : mean);
  return tiny ? r * 0x1p50f : r;
}

// The codes of four floats over 2^e, by the conversion instruction: the
// nearest code, the even one between two, at most 6 in size.
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], int e) {
  const float scale = __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
  const uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], scale, 0);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
}
// The largest m of the eight lanes of a block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, dpp_u<0xB1>(0u, m));
  m = max(m, dpp_u<0x4E>(0u, m));
  return max(m, dpp_u<0x141>(0u, m));
}
// Least E in [-126, 125] with amax <= 7 * 2^E (0 for amax == 0): with
// amax = f * 2^x, 1 <= f < 2, that is x - 2 for f <= 7/4 and x - 1 above.
__device__ __forceinline__ int block_exponent(bool zero, int x, bool above) {
  return zero ? 0 : min(max(x - 2 + (above ? 1 : 0), -126), 125);
}

// Four values as 16 bits of codes, and the scale byte of their block of 32.
__device__ __forceinline__ uint32_t quantise4(const float (&v)[4], uint32_t& scale) {
  uint32_t m = 0;
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = v[i] + 0.f;  // no -0, whose code has no sign
    m = max(m, __builtin_bit_cast(uint32_t, x[i]) & 0x7FFFFFFFu);
  }
  m = block_max(m);
  const int e = block_exponent(m == 0, (int)(m >> 23) - 127, (m & 0x7FFFFFu) > 0x600000u);
  scale = (uint32_t)(e + 127);
  return codes4(x, e);
}
// The same of 64-bit values, exactly: of a value's lower 32 bits it matters
// only whether there are any (the borders have at most three bits), so that a
// float of value / 2^e with that in its last bit falls on the same side of
// every border.
__device__ __forceinline__ uint32_t quantise4(const double (&v)[4], uint32_t& scale) {
  uint32_t h[4], m = 0;  // the upper 31 bits without the sign, then "and more"
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v[i]);
    h[i] = (uint32_t)(b >> 32) << 1 | ((uint32_t)b ? 1u : 0u);
    m = max(m, h[i]);
  }
  m = block_max(m);
  const int e = block_exponent(m == 0, (int)(m >> 21) - 1023, (m & 0x1FFFFFu) > 0x180000u);
  scale = (uint32_t)(e + 127);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 896 + e: from the exponent's offset of 1023 to 127, over 2^e.
    const int r = min(max((int)(h[i] >> 1) - ((896 + e) << 20), 0), (255 << 20) - 1);
    const uint32_t sign = h[i] ? (uint32_t)(__builtin_bit_cast(uint64_t, v[i]) >> 32) & 0x80000000u : 0u;
    x[i] = __builtin_bit_cast(float, (uint32_t)r << 3 | (h[i] & 1u) | sign);
  }
  return codes4(x, 0);
}

// N elements as they lie in memory, aligned as one element is: the memory
// path takes wide accesses at any address.
template <typename T, int N>
struct Raw {
  static constexpr int kWords = N * sizeof(T) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(w, p, sizeof(w)); }
  __device__ __forceinline__ void store(T* p) const { __builtin_memcpy(p, w, sizeof(w)); }
  // Past the caches (non-temporal).
  __device__ __forceinline__ void stream(T* p) const {
    typedef uint32_t Piece __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      __builtin_nontemporal_store(Piece{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]},
                                  reinterpret_cast<Piece*>(p) + i);
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, w[i]);
    else return (float)__builtin_bit_cast(T, (uint16_t)(i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu));
  }
  __device__ __forceinline__ void set(const float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __builtin_bit_cast(uint32_t, x[i]);
      else
        w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (T)x[2 * i]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (T)x[2 * i + 1]) << 16;
    }
  }
  __device__ __forceinline__ void scale(float by) {
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (*this)[i] * by;
    set(x);
  }
  // The neighbours swapped, where mask is set; 0 elsewhere.
  __device__ __forceinline__ void swap_of(const Raw& x, uint32_t mask) {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      w[i] = (sizeof(T) == 4 ? x.w[i ^ 1] : x.w[i] << 16 | x.w[i] >> 16) & mask;
  }
};

// A wave takes as many heads as it has room for at a time (a step): first the
// token's key/value heads, then its queries, kAhead steps at once; the
// workgroups of a token share its steps.
template <int D, typename T>
__global__ __launch_bounds__(kBlock) void k_kv_append(AppendArgs a) {
  constexpr int LG = query_lanes(D), kStep = kWave / LG, kAhead = 4 / sizeof(T);
  constexpr int KG = key_lanes(D), kKeyStep = kWave / KG;
  __shared__ __align__(16) Tables<D> tab;
  const int i = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const int lane = threadIdx.x & (kWave - 1), mine = lane / LG;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int c0 = 8 * (lane % LG), kc0 = 4 * (lane % KG), half = a.rotary / 2;
  const bool live = c0 < D, key_live = kc0 < D;
  // Whether a channel is turned with one apart, and where that lies from it.
  auto apart = [&](int c) { return c < a.rotary && !a.interleaved; };
  auto turn = [&](int c) { return c < half ? half : -half; };
  auto near = [&](int c) { return c < a.rotary ? ~0u : 0u; };  // of neighbours
  const int s_begin = part * a.steps_per_part;
  const int s_end = min(s_begin + a.steps_per_part, a.steps), k_end = min(a.k_steps, s_end);
  int sk = s_begin + wv;
  int s = sk + (max(k_end - sk, 0) + kWavesPerBlock - 1) / kWavesPerBlock * kWavesPerBlock;  // first of queries

  Raw<T, 4> kx{}, ky{}, kv{};
  Raw<T, 8> x[kAhead]{}, y[kAhead]{};
  auto load_keys = [&](int s) {
    const int u = s * kKeyStep + lane / KG;
    if (!key_live || u >= a.kv.Hk) return;
    const T* row = (const T*)a.k + i * a.ks + u * D + kc0;
    kx.load(row);
    if (apart(kc0)) ky.load(row + turn(kc0));
    kv.load((const T*)a.v + i * a.vs + u * D + kc0);
  };
  auto load_queries = [&](int s) {
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int at = s + n * kWavesPerBlock, u = (at - a.k_steps) * kStep + mine;
      if (at < s_end && live && u < a.kv.Hq) {
        const T* row = (const T*)a.q + i * a.qs + u * D + c0;
        x[n].load(row);
        if (apart(c0)) y[n].load(row + turn(c0));
      }
    }
  };
  // Asked for before anything else is known (a row of no sequence too, to drop it).
  if (sk < k_end) load_keys(sk);
  load_queries(s);

  const Pair pair(a, min((int)threadIdx.x, D / 2 - 1));
  double pos = a.positions ? (double)a.positions[i] : 0.0;

  const KvToken tok = kv_token(a.kv, i);
  if (tok.b < 0) return;
  if (!a.positions) pos = (double)tok.place;
  if (threadIdx.x < D / 2) pair.fill(tab, pos, s_begin < a.k_steps, s_end > a.k_steps);
  __syncthreads();

  for (; sk < k_end; sk += kWavesPerBlock) {
    const int u = sk * kKeyStep + lane / KG, sub = lane % KG;
    const bool on = key_live && u < a.kv.Hk;
    double k[4], r = 1.0;
    float v[4];
    if (a.interleaved) ky.swap_of(kx, near(kc0));
    if (a.k_norm) {
      double ss = 0.0;
#pragma unroll
      for (int e = 0; e < 4; ++e) ss += (double)kx[e] * (double)kx[e];
      r = 1.0 / sqrt(group_sum<KG>(ss) / D + (double)a.eps);
    }
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = key_live ? kc0 + e : e;
      k[e] = r * ((double)kx[e] * tab.ka[c] + (double)ky[e] * tab.kb[c]);
      v[e] = kv[e];
      bad |= !(fabs(k[e]) < INFINITY) || !(fabsf(v[e]) < INFINITY);
    }
    if (sk + kWavesPerBlock < k_end) load_keys(sk + kWavesPerBlock);
    const uint64_t unit = KG == kWave ? ~0ull : (1ull << KG) - 1;
    const bool nan_token = (__ballot(bad && on) >> (lane & ~(KG - 1))) & unit;
    uint32_t ke, ve;
    uint32_t kc = quantise4(k, ke), vc = quantise4(v, ve);
    if (nan_token) {
      kc = vc = 0;
      ke = 255;
      ve = 127;
    }
    // Two lanes' codes are a dword.
    kc |= dpp_u<0xB1>(0u, kc) << 16;
    vc |= dpp_u<0xB1>(0u, vc) << 16;
    const int64_t base = on ? kv_page_base(a.kv, tok.b, tok.place, u) : -1;
    if (base >= 0) {
      const int P = 1 << a.kv.page_shift, o = (int)(tok.place & (P - 1));
      uint8_t* c = a.cache + base;
      if (sub % 2 == 0) {
        *reinterpret_cast<uint32_t*>(c + o * (D / 2) + 2 * sub) = kc;
        *reinterpret_cast<uint32_t*>(c + (P + o) * (D / 2) + 2 * sub) = vc;
      }
      if (sub % 8 == 0) {
        c[P * D + o * (D / 32) + sub / 8] = (uint8_t)ke;
        c[P * D + (P + o) * (D / 32) + sub / 8] = (uint8_t)ve;
      }
    }
  }
  if (s >= s_end) return;

  float qa[8], qb[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    qa[e] = tab.qa[live ? c0 + e : e];
    qb[e] = tab.qb[live ? c0 + e : e];
  }
  T* out = (T*)a.q_out + (int64_t)i * a.kv.Hq * D + c0;
  for (; s < s_end; s += kAhead * kWavesPerBlock) {
    Raw<T, 8> z[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      if (a.interleaved) y[n].swap_of(x[n], near(c0));
      float t[8], r = 1.f;
      if (a.q_norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[n][e], x[n][e], ss);
        float mean = group_sum<LG>(ss) * (1.f / D) + a.eps;
        // Squares that pass the range of 32 bits: once more, of scaled channels.
        const bool huge = !(mean < 1e30f), tiny = mean < 1e-30f;
        if constexpr (!std::is_same_v<T, _Float16>)
          if (__ballot(huge || tiny)) {
            const float by = huge ? 0x1p-96f : tiny ? 0x1p96f : 1.f;
            x[n].scale(by);
            y[n].scale(by);
            ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[n][e], x[n][e], ss);
            mean = group_sum<LG>(ss) * (1.f / D) + a.eps * by * by;
          }
        r = norm_factor(mean);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = r * fmaf(x[n][e], qa[e], y[n][e] * qb[e]);
      z[n].set(t);
    }
    load_queries(s + kAhead * kWavesPerBlock);
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int at = s + n * kWavesPerBlock, u = (at - a.k_steps) * kStep + mine;
      if (at < s_end && live && u < a.kv.Hq) z[n].stream(out + u * D);
    }
  }
}

struct ReadArgs {
  KvArgs kv;
  const uint8_t* cache;
  float *k_out, *v_out;
};

// One lane takes eight channels of one row and head.
__global__ __launch_bounds__(kBlock) void k_kv_read(ReadArgs a) {
  const int D = a.kv.D, per_row = a.kv.Hk * (D / 8);
  const int blocks = (per_row + kBlock - 1) / kBlock;
  const int i = blockIdx.x / blocks;
  const int w = (blockIdx.x % blocks) * kBlock + threadIdx.x;
  const KvToken tok = kv_token(a.kv, i);
  if (tok.b < 0 || w >= per_row) return;
  const int h = w / (D / 8), sub = w % (D / 8);
  const int64_t base = kv_page_base(a.kv, tok.b, tok.place, h);
  const int P = 1 << a.kv.page_shift, o = (int)(tok.place & (P - 1));
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    float* out = side ? a.v_out : a.k_out;
    if (!out) continue;
    float x[8] = {};
    if (base >= 0) {
      const uint8_t* c = a.cache + base;
      const uint32_t word = *reinterpret_cast<const uint32_t*>(c + (side * P + o) * (D / 2) + 4 * sub);
      const uint32_t e = c[P * D + (side * P + o) * (D / 32) + sub / 4];
      // 2^(e - 127), its lowest value below the normal floats; 255 is NaN.
      const float s = e == 255 ? NAN : __builtin_bit_cast(float, e ? e << 23 : 0x00400000u);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const uint32_t m = (word >> (4 * n)) & 7;
        // E2M1 magnitude: (2 + fraction) * 2^(exponent - 2), below 1 a plain half.
        const float mag = m < 2 ? 0.5f * (float)m : (float)((2 | (m & 1)) << (m >> 1)) * 0.25f;
        x[n] = ((word >> (4 * n)) & 8 ? -mag : mag) * s;
      }
    }
    Raw<float, 8> raw;
    raw.set(x);
    raw.stream(out + ((int64_t)i * a.kv.Hk + h) * D + 8 * sub);
  }
}

template <int D>
void launch_append(const AppendArgs& a, int32_t dtype, int grid, hipStream_t st) {
  switch (dtype) {
    case MOE_F32: hipLaunchKernelGGL((k_kv_append<D, float>), dim3(grid), dim3(kBlock), 0, st, a); break;
    case MOE_BF16: hipLaunchKernelGGL((k_kv_append<D, bf16>), dim3(grid), dim3(kBlock), 0, st, a); break;
    default: hipLaunchKernelGGL((k_kv_append<D, _Float16>), dim3(grid), dim3(kBlock), 0, st, a); break;
  }
}

}  // namespace
}  // namespace svr

using namespace svr;

extern "C" {

int32_t moe_kv_cache_bytes(const moe_kv_desc* desc, int64_t n_pages, int64_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const int32_t rc = kv_check_desc(desc);
  if (rc != MOE_OK) return rc;
  if (n_pages < 1 || n_pages > INT32_MAX) return MOE_ERR_SHAPE;
  *bytes = n_pages * desc->n_kv_heads * kv_page_bytes(desc);
  return MOE_OK;
}

int32_t moe_kv_append(const moe_kv_desc* desc, const moe_kv_batch* batch, int32_t dtype,
                      const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const void* v, int64_t v_stride, const float* q_norm, const float* k_norm,
                      const float* inv_freq, const int32_t* positions, void* cache,
                      int32_t n_pages, void* q_out, void* hip_stream) {
  int32_t rc = kv_check_desc(desc);
  if (rc == MOE_OK) rc = kv_check_batch(desc, batch, true);
  if (rc != MOE_OK) return rc;
  const int es = kv_elem_size(dtype);
  if (!es) return MOE_ERR_DTYPE;
  const int D = desc->head_dim;
  if (n_pages < 1) return MOE_ERR_SHAPE;
  if (batch->n_tokens == 0 || batch->n_seqs == 0) return MOE_OK;
  if (!k || !v || !cache || (q == nullptr) != (q_out == nullptr)) return MOE_ERR_NULL;
  if (desc->rotary_dims > 0 && !inv_freq) return MOE_ERR_NULL;
  if ((q && q_stride < (int64_t)desc->n_heads * D) || k_stride < (int64_t)desc->n_kv_heads * D ||
      v_stride < (int64_t)desc->n_kv_heads * D)
    return MOE_ERR_SHAPE;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out) % es) return MOE_ERR_ARG;
  if (((uintptr_t)q_norm | (uintptr_t)k_norm | (uintptr_t)inv_freq | (uintptr_t)positions) % 4)
    return MOE_ERR_ARG;
  if ((uintptr_t)cache % 16) return MOE_ERR_ARG;

  AppendArgs a{};
  a.kv = kv_args(desc, batch, n_pages);
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.cache = (uint8_t*)cache;
  a.q_out = q_out;
  a.eps = desc->norm_eps;
  a.rotary = desc->rotary_dims;
  a.interleaved = desc->flags & MOE_KV_ROTARY_INTERLEAVED;
  // One workgroup a token where there are tokens enough to fill the chip (five
  // workgroups a CU), several, down to a step a wave, where there are not.
  const int step = kWave / query_lanes(D), key_step = kWave / key_lanes(D);
  a.k_steps = (desc->n_kv_heads + key_step - 1) / key_step;
  a.steps = a.k_steps + (q ? (desc->n_heads + step - 1) / step : 0);
  const int want = (1280 + batch->n_tokens - 1) / batch->n_tokens;
  const int rounds = (a.steps + want * kWavesPerBlock - 1) / (want * kWavesPerBlock);
  a.steps_per_part = rounds * kWavesPerBlock;
  a.parts = (a.steps + a.steps_per_part - 1) / a.steps_per_part;
  const int grid = batch->n_tokens * a.parts;
  hipStream_t st = (hipStream_t)hip_stream;
  (void)hipGetLastError();
  switch (D) {
    case 64: launch_append<64>(a, dtype, grid, st); break;
    case 128: launch_append<128>(a, dtype, grid, st); break;
    case 192: launch_append<192>(a, dtype, grid, st); break;
    default: launch_append<256>(a, dtype, grid, st); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

int32_t moe_kv_read(const moe_kv_desc* desc, const moe_kv_batch* batch, const void* cache,
                    int32_t n_pages, float* k_out, float* v_out, void* hip_stream) {
  int32_t rc = kv_check_desc(desc);
  if (rc == MOE_OK) rc = kv_check_batch(desc, batch, true);
  if (rc != MOE_OK) return rc;
  if (n_pages < 1) return MOE_ERR_SHAPE;
  if (batch->n_tokens == 0 || batch->n_seqs == 0) return MOE_OK;
  if (!cache || (!k_out && !v_out)) return MOE_ERR_NULL;
  if ((uintptr_t)cache % 16 || ((uintptr_t)k_out | (uintptr_t)v_out) % 4) return MOE_ERR_ARG;
  const int per_row = desc->n_kv_heads * (desc->head_dim / 8);
  const int64_t grid = (int64_t)batch->n_tokens * ((per_row + kBlock - 1) / kBlock);
  if (!kv_grid_fits(grid, kBlock)) return MOE_ERR_SHAPE;
  ReadArgs a{};
  a.kv = kv_args(desc, batch, n_pages);
  a.cache = (const uint8_t*)cache;
  a.k_out = k_out;
  a.v_out = v_out;
  (void)hipGetLastError();
  hipLaunchKernelGGL(k_kv_read, dim3((unsigned)grid), dim3(kBlock), 0, (hipStream_t)hip_stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
