// The gated grouped product and its gradient for f32 operands and outputs.
#include "gl_glu_tile.hpp"

namespace gl {

hipError_t launch_glu_f32(const GluParams &p, bool grad, hipStream_t s) {
  return grad ? launch_glu<IN_F32, EL_F32, EPI_GLU_GRAD>(p, s) : launch_glu<IN_F32, EL_F32, EPI_GLU>(p, s);
}

}  // namespace gl
