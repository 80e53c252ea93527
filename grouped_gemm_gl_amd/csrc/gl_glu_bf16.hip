// The gated grouped product and its gradient for bf16 operands and outputs.
#include "gl_glu_tile.hpp"

namespace gl {

hipError_t launch_glu_bf16(const GluParams &p, bool grad, hipStream_t s) {
  return grad ? launch_glu<IN_BF16, EL_BF16, EPI_GLU_GRAD>(p, s) : launch_glu<IN_BF16, EL_BF16, EPI_GLU>(p, s);
}

}  // namespace gl
