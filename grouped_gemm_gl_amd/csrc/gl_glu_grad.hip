// The gradient of a gated activation from the kept values h [T, 2F]: with g and u the halves of
// a row of h, dh = [da u act'(g), da act(g)], and on request a = act(g) u again (the next
// layer's input, where the forward's was not kept).
//
// HBM-bound elementwise work: each thread moves 16 bytes of each operand, all in fp32, one
// rounding per output.  Per row it reads 3F and writes 2F (3F) elements: 4099 rows, F 1400 fp16, 13.2 us,
// 4.3 TB/s.
#include "gl_glu.hpp"

namespace gl {

constexpr int kGradThreads = 256;

template <int EL>
__global__ __launch_bounds__(kGradThreads) void glu_grad_kernel(const char *h, const char *__restrict__ da,
                                                                int64_t F, int64_t n, int act, char *dh,
                                                                char *__restrict__ a) {
  using V = Vec<EL>;
  constexpr int B = elem_bytes(EL);
  const int64_t per_row = F / V::n;
  for (int64_t t = (int64_t)blockIdx.x * kGradThreads + threadIdx.x; t < n; t += (int64_t)gridDim.x * kGradThreads) {
    const int64_t r = t / per_row, c = (t - r * per_row) * V::n;
    float g[V::n], u[V::n], d[V::n], o[V::n];
    V::load(h + (r * 2 * F + c) * B, g);
    V::load(h + (r * 2 * F + F + c) * B, u);
    V::load(da + (r * F + c) * B, d);
    with_activation(act, [&](auto tag) {
#pragma unroll
      for (int i = 0; i < V::n; ++i) {
        float slope;
        const float y = activate<true, decltype(tag)::value>(g[i], slope);
        o[i] = y * u[i];
        g[i] = d[i] * u[i] * slope;
        u[i] = d[i] * y;
      }
    });
    V::store(dh + (r * 2 * F + c) * B, g);
    V::store(dh + (r * 2 * F + F + c) * B, u);
    if (a) V::store(a + (r * F + c) * B, o);
  }
}

// dh may be h: a thread reads both halves' values before it writes them.
hipError_t launch_glu_grad(int el, int64_t T, int64_t F, int act, const void *h, const void *da, void *dh, void *a,
                           hipStream_t s) {
  const int64_t n = T * (F / (el == EL_F32 ? 4 : 8));
  if (n == 0) return hipSuccess;
  const int64_t blocks = (n + kGradThreads - 1) / kGradThreads, most = kSliceThreads / kGradThreads;
  const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(kGradThreads);
  const char *hp = (const char *)h, *dp = (const char *)da;
  if (el == EL_F32)
    hipLaunchKernelGGL(glu_grad_kernel<EL_F32>, grid, block, 0, s, hp, dp, F, n, act, (char *)dh, (char *)a);
  else if (el == EL_F16)
    hipLaunchKernelGGL(glu_grad_kernel<EL_F16>, grid, block, 0, s, hp, dp, F, n, act, (char *)dh, (char *)a);
  else
    hipLaunchKernelGGL(glu_grad_kernel<EL_BF16>, grid, block, 0, s, hp, dp, F, n, act, (char *)dh, (char *)a);
  return hipGetLastError();
}

}  // namespace gl
