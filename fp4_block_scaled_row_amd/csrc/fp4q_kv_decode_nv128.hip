// fp4q_kv_decode_nv128.hip -- the few-row attention kernels of NVFP4, head_dim 128.
#include "fp4q_kv_decode.h"
#include "fp4q_kv_dispatch.h"

namespace fp4q {
hipError_t launch_decode_nv128(const KvAttendLaunch& a, int tiles, int cus, hipStream_t st) {
  return launch_decode_d<128, 1>(a, tiles, cus, st);
}
}  // namespace fp4q
