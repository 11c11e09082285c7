// A wave's tile of a row of logits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace svr {

constexpr int kTileCols = 16;                  // columns of a lane in a tile
constexpr int kRowTile = kTileCols * kWave;    // columns of a wave's tile

// 16 columns of a lane: pieces of 16 bytes, lane after lane.  Kept as the
// words they come in: as elements, the compiler takes 16-bit ones apart where
// they are loaded, and waits for them there.
template <typename T>
struct RowTile {
  static constexpr int kElems = 16 / sizeof(T);  // of a piece
  static constexpr int kPieces = kTileCols / kElems;
  uint32_t w[4 * kPieces];

  // Of the tile at column base, past the caches; columns from V on are -inf.
  // (The memory path takes 16 bytes at any address.)
  __device__ __forceinline__ void load(const T* row, int base, int V, int lane) {
    const T* at = row + base + lane * kElems;
    if (base + kRowTile <= V) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        typedef uint32_t Four __attribute__((ext_vector_type(4), aligned(2)));
        const Four q = __builtin_nontemporal_load(reinterpret_cast<const Four*>(at + p * (kElems * kWave)));
        __builtin_memcpy(w + 4 * p, &q, 16);
      }
    } else {
      T x[kTileCols];
#pragma unroll
      for (int e = 0; e < kTileCols; ++e) {
        const int c = (e / kElems) * (kElems * kWave) + e % kElems;
        x[e] = base + lane * kElems + c < V ? at[c] : (T)-INFINITY;
      }
      __builtin_memcpy(w, x, sizeof(x));
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4 * kPieces; ++i) w[i] = 0;
  }
  // Whole words up to here, and waited for here.
  __device__ __forceinline__ void arrive() {
#pragma unroll
    for (int i = 0; i < 4 * kPieces; ++i) asm("" : "+v"(w[i]));
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, w[e]);
    else return (float)__builtin_bit_cast(T, (uint16_t)(e % 2 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu));
  }
};

}  // namespace svr
