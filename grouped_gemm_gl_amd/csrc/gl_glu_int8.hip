// The grouped product of 8-bit integers with scales for each token and channel, plain and gated,
// and the rows' quantizer.
//
// quantize_int8: scale = m / 127 and q = rint(v * (127 * (1 / m))) with m the row's largest magnitude,
// at least 2^-100 (so neither quotient overflows and scale is normal), every operation rounded once in
// fp32.  1 / m is subnormal for m past 2^126, so subnormals are not to be flushed; it keeps 21 bits or more there.
// A row with an infinity or NaN gets codes 0 and scale NaN, so that whatever is multiplied with it is NaN.
// HBM-bound: a workgroup a row, read twice, the second time from cache: 16384 rows of 4096 bf16 in 41 us,
// 4.9 TB/s, the rate of a copy; four rows in the time of a launch.  Rows of fewer than 2048 values leave threads
// without any: 131072 rows of 768 126 us, 2.4 TB/s, of 128 81 us, 0.6 TB/s.
#include "gl_glu_tile.hpp"

namespace gl {

template <int EPI>
static hipError_t launch_int8(int el_out, const GluParams &p, hipStream_t s) {
  if (el_out == EL_F32) return launch_glu<IN_I8, EL_F32, EPI>(p, s);
  if (el_out == EL_F16) return launch_glu<IN_I8, EL_F16, EPI>(p, s);
  return launch_glu<IN_I8, EL_BF16, EPI>(p, s);
}

hipError_t launch_glu_int8(int el_out, const GluParams &p, bool gated, hipStream_t s) {
  return gated ? launch_int8<EPI_GLU>(el_out, p, s) : launch_int8<EPI_PLAIN>(el_out, p, s);
}

constexpr int kQiThreads = 256;

template <int EL>
__global__ __launch_bounds__(kQiThreads) void quantize_int8_kernel(const char *__restrict__ src, int64_t rows,
                                                                   int64_t cols, int8_t *__restrict__ data,
                                                                   float *__restrict__ scale) {
  using V = Vec<EL>;
  __shared__ float s_max[kQiThreads / 64];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const char *row = src + r * cols * elem_bytes(EL);
    uint32_t m = 0;  // magnitudes as bits order like the values, infinities and NaN above all
    for (int64_t c = threadIdx.x * V::n; c < cols; c += kQiThreads * V::n) {
      float v[V::n];
      V::load(row + c * elem_bytes(EL), v);
#pragma unroll
      for (int i = 0; i < V::n; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = __uint_as_float(m);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQiThreads / 64; ++i) m = max(m, __float_as_uint(s_max[i]));
    __syncthreads();
    const bool finite = m < 0x7f800000u;
    const float top = fmaxf(__uint_as_float(m), 0x1p-100f);
    const float inv = finite ? 127.f * (1.f / top) : 0.f;
    for (int64_t c = threadIdx.x * V::n; c < cols; c += kQiThreads * V::n) {
      float v[V::n];
      V::load(row + c * elem_bytes(EL), v);
      uint32_t o[V::n / 4];
#pragma unroll
      for (int i = 0; i < V::n; i += 4) {
        uint32_t word = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) word |= (uint32_t)((finite ? (int)rintf(v[i + k] * inv) : 0) & 0xff) << (8 * k);
        o[i / 4] = word;
      }
#pragma unroll
      for (int i = 0; i < V::n / 4; ++i) *(uint32_t *)(data + r * cols + c + 4 * i) = o[i];
    }
    if (threadIdx.x == 0) scale[r] = finite ? top / 127.f : __uint_as_float(0x7fc00000u);
  }
}

hipError_t launch_quantize_int8(int el, int64_t rows, int64_t cols, const void *src, int8_t *data, float *scale,
                                hipStream_t s) {
  const dim3 grid((unsigned)(rows < (1 << 20) ? rows : 1 << 20)), block(kQiThreads);
  const char *x = (const char *)src;
  if (el == EL_F32)
    hipLaunchKernelGGL(quantize_int8_kernel<EL_F32>, grid, block, 0, s, x, rows, cols, data, scale);
  else if (el == EL_F16)
    hipLaunchKernelGGL(quantize_int8_kernel<EL_F16>, grid, block, 0, s, x, rows, cols, data, scale);
  else
    hipLaunchKernelGGL(quantize_int8_kernel<EL_BF16>, grid, block, 0, s, x, rows, cols, data, scale);
  return hipGetLastError();
}

}  // namespace gl
