// fp4q_linear_many_back_nv.hip -- instances of the tile kernel (see
// fp4q_linear_many.h): dx = dy W, weights in NVFP4.
#include "fp4q_linear_many.h"

namespace fp4q {

hipError_t launch_many_back_nv(const ManyArgs& a, int size, hipStream_t s) {
  return a.l.x_type == kXF32 ? launch_many_size<1, kXF32, kTransposed>(a, size, s)
                             : launch_many_size<1, kXBF16, kTransposed>(a, size, s);
}

}  // namespace fp4q
