// Attention kernels of head size 64 (a translation unit of its own: the families compile in parallel).
#include "launch_attention.h"

namespace svr {
template int32_t launch_kv_attention<64>(const AttnArgs&, int32_t, int, int, int, hipStream_t);
}  // namespace svr
