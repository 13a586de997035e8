// fp4q_linear_many_mx.hip -- instances of the tile kernel (see
// fp4q_linear_many.h): y = x W^T and the gated form, weights in MXFP4.
#include "fp4q_linear_many.h"

namespace fp4q {

hipError_t launch_many_mx(const ManyArgs& a, int size, hipStream_t s) {
  switch (a.l.x_type * 2 + a.l.gated) {
    case 0: return launch_many_size<0, kXF32, kForward>(a, size, s);
    case 1: return launch_many_size<0, kXF32, kGated>(a, size, s);
    case 2: return launch_many_size<0, kXBF16, kForward>(a, size, s);
    case 3: return launch_many_size<0, kXBF16, kGated>(a, size, s);
    case 4: return launch_many_size<0, kXE4M3, kForward>(a, size, s);
    case 5: return launch_many_size<0, kXE4M3, kGated>(a, size, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace fp4q
