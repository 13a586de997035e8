// fp4q_kv_prefill_nv96.hip -- the many-row attention kernels of NVFP4, head_dim 96.
#include "fp4q_kv_prefill.h"
#include "fp4q_kv_dispatch.h"

namespace fp4q {
hipError_t launch_prefill_nv96(const KvAttendLaunch& a, int waves, int cus, hipStream_t st) {
  return launch_prefill_d<96, 1>(a, waves, cus, st);
}
}  // namespace fp4q
