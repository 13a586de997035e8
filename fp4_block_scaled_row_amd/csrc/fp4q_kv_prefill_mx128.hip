// fp4q_kv_prefill_mx128.hip -- the many-row attention kernels of MXFP4, head_dim 128.
#include "fp4q_kv_prefill.h"
#include "fp4q_kv_dispatch.h"

namespace fp4q {
hipError_t launch_prefill_mx128(const KvAttendLaunch& a, int waves, int cus, hipStream_t st) {
  return launch_prefill_d<128, 0>(a, waves, cus, st);
}
}  // namespace fp4q
