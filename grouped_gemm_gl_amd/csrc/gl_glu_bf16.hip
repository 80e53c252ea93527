// The gated grouped product and its gradient for bf16 operands and outputs, and the products of its
// backward on small tiles.
#include "gl_glu_back.hpp"
#include "gl_glu_tile.hpp"

namespace gl {

hipError_t launch_glu_bf16(const GluParams &p, bool grad, hipStream_t s) {
  return grad ? launch_glu<IN_BF16, EL_BF16, EPI_GLU_GRAD>(p, s) : launch_glu<IN_BF16, EL_BF16, EPI_GLU>(p, s);
}

hipError_t launch_glu_back_bf16(const BackParams &p, bool wgrad, bool out_f32, hipStream_t s) {
  return launch_glu_back<IN_BF16, EL_BF16>(p, wgrad, out_f32, s);
}

}  // namespace gl
