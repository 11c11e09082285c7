// One instance family of the attention kernel: every row tile and type of a head size.
#pragma once

#include "kv_attention.h"

namespace svr {

template <int D>
int32_t launch_kv_attention(const AttnArgs& a, int32_t dtype, int row_tiles, int waves, int grid,
                            hipStream_t st) {
  const dim3 n(grid), t(waves * kWave);
#define SVR_ATTN(RT, NT, W, T)                                                          \
  if constexpr (RT <= attn_most_row_tiles(D, NT)) {                                     \
    if (row_tiles == RT && waves == W)                                                  \
      hipLaunchKernelGGL((k_kv_attention<D, RT, NT, W, T>), n, t, 0, st, a);            \
  }
  if (dtype == MOE_BF16) {
    SVR_ATTN(1, 1, kAttnWaves, bf16)
    SVR_ATTN(2, 1, kAttnWaves, bf16)
    SVR_ATTN(2, 1, kAttnPartWaves, bf16)
  } else if (dtype == MOE_F16) {
    SVR_ATTN(1, 2, kAttnWaves, _Float16)
    SVR_ATTN(2, 2, kAttnWaves, _Float16)
    SVR_ATTN(2, 2, kAttnPartWaves, _Float16)
  } else {
    SVR_ATTN(1, 3, kAttnWaves, float)
    SVR_ATTN(2, 3, kAttnWaves, float)
    SVR_ATTN(2, 3, kAttnPartWaves, float)
  }
#undef SVR_ATTN
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // namespace svr
