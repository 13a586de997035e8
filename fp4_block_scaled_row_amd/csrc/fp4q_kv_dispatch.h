// fp4q_kv_dispatch.h -- the attention kernels' launchers, one translation unit
// per format and head_dim.
#pragma once

#include "fp4q_kv.h"

namespace fp4q {
#define FP4Q_KV_LAUNCHERS(X)                                                                       \
  hipError_t launch_decode_##X(const KvAttendLaunch& a, int tiles, int cus, hipStream_t st); \
  hipError_t launch_prefill_##X(const KvAttendLaunch& a, int waves, int cus, hipStream_t st)
FP4Q_KV_LAUNCHERS(mx64);
FP4Q_KV_LAUNCHERS(mx96);
FP4Q_KV_LAUNCHERS(mx128);
FP4Q_KV_LAUNCHERS(mx256);
FP4Q_KV_LAUNCHERS(nv64);
FP4Q_KV_LAUNCHERS(nv96);
FP4Q_KV_LAUNCHERS(nv128);
FP4Q_KV_LAUNCHERS(nv256);
#undef FP4Q_KV_LAUNCHERS
}  // namespace fp4q
