// Head norms, position rotation and append to the paged 4-bit cache, and
// reading rows back (include/moe_kv.h).
//
// A unit is one head vector: a query head, or a key head with its value head
// (together, so that a NaN or infinity in either marks the token).  A group
// of LG lanes takes a unit, eight channels a lane: one 16-byte load of a
// 16-bit type, a 4-bit block of 32 channels is four lanes, and a lane's
// codes are one dword.  The pair of a rotated channel is in the same lane
// (neighbours) or a fixed number of lanes away.
//
// The pass is bound by its bytes: each of q, k, v is read once, q_out and
// the codes written once.  A workgroup serves one token, so that the angles
// (64-bit: at place 60000 a 32-bit angle is off by 2^-9 of a turn's radian)
// are taken once for all heads; queries are normed and rotated in 32 bits,
// keys in 64, because a code is a whole number and a key next to a rounding
// border must fall on its own side whatever the order of the sum.
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
  int rotary, interleaved, units_per_block, vec;
};

template <int D>
struct Group {
  static constexpr int kLanes = D <= 64 ? 8 : D <= 128 ? 16 : 32;  // lanes of a unit
  static constexpr int kUnits = kBlock / kLanes;                   // units of a pass
};

template <typename F, int LG>
__device__ __forceinline__ F group_sum(F v) {
#pragma unroll
  for (int m = 1; m < LG; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// x[8] (channels c0..c0+7 of one head) normed and rotated in F.
template <typename F, int LG>
__device__ __forceinline__ void norm_rotate(const AppendArgs& a, int D, int sub, bool live,
                                            const float* w, const double2* cs, F (&x)[8]) {
  const int c0 = 8 * sub;
  if (w) {
    F ss = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
    ss = group_sum<F, LG>(ss);
    const F r = (F)1 / sqrt(ss / (F)D + (F)a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (F)(live ? w[c0 + i] : 0.f);
  }
  if (a.rotary == 0) return;
  if (a.interleaved) {
    if (c0 < a.rotary) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double2 t = cs[c0 / 2 + i];
        const F p = x[2 * i], n = x[2 * i + 1];
        x[2 * i] = p * (F)t.x - n * (F)t.y;
        x[2 * i + 1] = n * (F)t.x + p * (F)t.y;
      }
    }
    return;
  }
  const int half = a.rotary / 2;  // a multiple of 8: the pair is half / 8 lanes away
  const bool first = c0 < half;
  const int other = (int)(threadIdx.x & (kWave - 1)) + (first ? half / 8 : -(half / 8));
  F y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __shfl(x[i], other & (kWave - 1), kWave);
  if (c0 < a.rotary) {
    const int j = first ? c0 : c0 - half;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double2 t = cs[j + i];
      x[i] = first ? x[i] * (F)t.x - y[i] * (F)t.y : x[i] * (F)t.x + y[i] * (F)t.y;
    }
  }
}

// Least E in [-126, 125] with amax <= 7 * 2^E (0 for amax == 0): with
// amax = f * 2^x, 1 <= f < 2, that is x - 2 for f <= 7/4 and x - 1 above.
__device__ __forceinline__ int block_exponent(double amax) {
  const uint64_t b = __builtin_bit_cast(uint64_t, amax);
  const int x = (int)(b >> 52) - 1023;
  const int e = x - 2 + ((b & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0);
  return amax == 0 ? 0 : min(max(e, -126), 125);
}
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t b = __builtin_bit_cast(uint32_t, amax);
  const int x = (int)(b >> 23) - 127;
  const int e = x - 2 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax == 0 ? 0 : min(max(e, -126), 125);
}
__device__ __forceinline__ double pow2(double, int e) {
  return __builtin_bit_cast(double, (uint64_t)(1023 + e) << 52);
}
__device__ __forceinline__ float pow2(float, int e) {
  return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
}

// Eight values as one dword of codes; the scale byte of their block of 32.
// The thresholds are the midpoints of the code values, each open on the side
// of the even code, so the result is exact for whatever x is.
template <typename F>
__device__ __forceinline__ uint32_t quantise8(const F (&x)[8], uint32_t& scale) {
  F amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmax(amax, fabs(x[i]));
  amax = fmax(amax, __shfl_xor(amax, 1, kWave));
  amax = fmax(amax, __shfl_xor(amax, 2, kWave));
  const int e = block_exponent(amax);
  const F inv = pow2((F)0, -e);
  scale = (uint32_t)(e + 127);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const F t = fabs(x[i]) * inv;
    uint32_t c = (t > (F)0.25) + (t >= (F)0.75) + (t > (F)1.25) + (t >= (F)1.75) +
                 (t > (F)2.5) + (t >= (F)3.5) + (t > (F)5.0);
    c |= x[i] < 0 ? 8u : 0u;
    word |= c << (4 * i);
  }
  return word;
}

template <int D, typename T>
__global__ __launch_bounds__(kBlock) void k_kv_append(AppendArgs a) {
  constexpr int LG = Group<D>::kLanes;
  __shared__ double2 s_cs[D / 2];
  const int blocks = (a.kv.Hq * (a.q ? 1 : 0) + a.kv.Hk + a.units_per_block - 1) / a.units_per_block;
  const int i = blockIdx.x / blocks, part = blockIdx.x % blocks;
  const int b = kv_sequence_of(a.kv, i);
  if (b < 0) return;
  const int64_t place = (int64_t)a.kv.lens[b] - a.kv.offs[b + 1] + i;
  if (a.rotary) {
    const double pos = a.positions ? (double)a.positions[i] : (double)place;
    for (int j = threadIdx.x; j < a.rotary / 2; j += kBlock) {
      double sn, cn;
      sincos(pos * (double)a.inv_freq[j], &sn, &cn);
      s_cs[j] = make_double2(cn, sn);
    }
    __syncthreads();
  }
  const int lane = threadIdx.x & (kWave - 1);
  const int sub = lane % LG;
  const bool live = 8 * sub < D;
  const int units = a.kv.Hk + (a.q ? a.kv.Hq : 0);
  const int u_end = min((part + 1) * a.units_per_block, units);
  // Whole passes, so that every lane takes part in the exchanges.
  for (int u0 = part * a.units_per_block; u0 < u_end; u0 += Group<D>::kUnits) {
    const int u = u0 + (int)threadIdx.x / LG;
    const bool on = live && u < u_end;
    if (u < a.kv.Hk) {
      float xf[8] = {}, v[8] = {};
      if (on) {
        load8((const T*)a.k + i * a.ks + (int64_t)u * D + 8 * sub, a.vec & 2, xf);
        load8((const T*)a.v + i * a.vs + (int64_t)u * D + 8 * sub, a.vec & 4, v);
      }
      double x[8];
      bool bad = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (double)xf[e];
      norm_rotate<double, LG>(a, D, sub, live, a.k_norm, s_cs, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) bad |= !(fabs(x[e]) < INFINITY) || !(fabsf(v[e]) < INFINITY);
      const uint64_t group = LG == 64 ? ~0ull : (1ull << LG) - 1;
      const bool nan_token = (__ballot(bad) >> (lane & ~(LG - 1))) & group;
      uint32_t ke, ve;
      uint32_t kw = quantise8(x, ke), vw = quantise8(v, ve);
      if (nan_token) {
        kw = vw = 0;
        ke = 255;
        ve = 127;
      }
      const int64_t base = on ? kv_page_base(a.kv, b, place, u) : -1;
      if (base >= 0) {
        const int P = 1 << a.kv.page_shift, o = (int)(place & (P - 1));
        uint8_t* c = a.cache + base;
        *reinterpret_cast<uint32_t*>(c + o * (D / 2) + 4 * sub) = kw;
        *reinterpret_cast<uint32_t*>(c + (P + o) * (D / 2) + 4 * sub) = vw;
        if (sub % 4 == 0) {
          c[P * D + o * (D / 32) + sub / 4] = (uint8_t)ke;
          c[P * D + (P + o) * (D / 32) + sub / 4] = (uint8_t)ve;
        }
      }
    } else {
      const int h = u - a.kv.Hk;
      float x[8] = {};
      if (on) load8((const T*)a.q + i * a.qs + (int64_t)h * D + 8 * sub, a.vec & 1, x);
      norm_rotate<float, LG>(a, D, sub, live, a.q_norm, s_cs, x);
      if (on) store8((T*)a.q_out + ((int64_t)i * a.kv.Hq + h) * D + 8 * sub, a.vec & 8, x);
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
  const int b = kv_sequence_of(a.kv, i);
  if (b < 0 || w >= per_row) return;
  const int64_t place = (int64_t)a.kv.lens[b] - a.kv.offs[b + 1] + i;
  const int h = w / (D / 8), sub = w % (D / 8);
  const int64_t base = kv_page_base(a.kv, b, place, h);
  const int P = 1 << a.kv.page_shift, o = (int)(place & (P - 1));
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
    store8(out + ((int64_t)i * a.kv.Hk + h) * D + 8 * sub, (uintptr_t)out % 16 == 0, x);
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
  auto aligned = [&](const void* p, int64_t stride) {
    return (uintptr_t)p % 16 == 0 && stride * es % 16 == 0;
  };
  a.vec = (aligned(q, q_stride) ? 1 : 0) | (aligned(k, k_stride) ? 2 : 0) |
          (aligned(v, v_stride) ? 4 : 0) | (aligned(q_out, 0) ? 8 : 0);
  const int units = desc->n_kv_heads + (q ? desc->n_heads : 0);
  const int pass = kBlock / (D <= 64 ? 8 : D <= 128 ? 16 : 32);
  a.units_per_block = pass;
  const int grid = batch->n_tokens * ((units + a.units_per_block - 1) / a.units_per_block);
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
  ReadArgs a{};
  a.kv = kv_args(desc, batch, n_pages);
  a.cache = (const uint8_t*)cache;
  a.k_out = k_out;
  a.v_out = v_out;
  const int per_row = desc->n_kv_heads * (desc->head_dim / 8);
  const int grid = batch->n_tokens * ((per_row + kBlock - 1) / kBlock);
  (void)hipGetLastError();
  hipLaunchKernelGGL(k_kv_read, dim3(grid), dim3(kBlock), 0, (hipStream_t)hip_stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
