// The gated grouped product and its gradient for f16 operands and outputs.
#include "gl_glu_tile.hpp"

namespace gl {

hipError_t launch_glu_f16(const GluParams &p, bool grad, hipStream_t s) {
  return grad ? launch_glu<IN_F16, EL_F16, EPI_GLU_GRAD>(p, s) : launch_glu<IN_F16, EL_F16, EPI_GLU>(p, s);
}

}  // namespace gl
