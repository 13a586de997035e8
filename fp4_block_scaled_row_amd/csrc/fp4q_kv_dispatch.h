// fp4q_kv_dispatch.h -- the attention kernels' launchers, one translation unit
// per format and head_dim.
#pragma once

#include "fp4q_kv.h"

namespace fp4q {
#define FP4Q_KV_DECODE(X) hipError_t launch_decode_##X(const KvAttendLaunch& a, int tiles, int cus, hipStream_t st)
FP4Q_KV_DECODE(mx64);
FP4Q_KV_DECODE(mx96);
FP4Q_KV_DECODE(mx128);
FP4Q_KV_DECODE(mx256);
FP4Q_KV_DECODE(nv64);
FP4Q_KV_DECODE(nv96);
FP4Q_KV_DECODE(nv128);
FP4Q_KV_DECODE(nv256);
#undef FP4Q_KV_DECODE
}  // namespace fp4q
