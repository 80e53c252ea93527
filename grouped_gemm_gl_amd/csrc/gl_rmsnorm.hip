// RMS norm with the residual's addition, its output in the layer's type and / or in
// MXFP8 codes, and its backward.
//
//   forward   s = x + r (fp32), h = round(s),
//             y = s * rstd * gamma with rstd = (mean(s^2) + eps)^-1/2 over the row
//   backward  xh = h * rstd, v = dy * gamma, c = mean(v * xh)
//             dx = dh + rstd * (v - xh * c),  dgamma = sum over rows of dy * xh
//
// The sum s stays in fp32 for the norm; h, y and the codes are each rounded once from
// fp32 values.  The backward takes rstd of the h it is given, so it is the gradient of
// the norm at exactly that h and no statistics are kept between the two.
#include <type_traits>

#include "gl_mx.hpp"
#include "gl_vec.hpp"

namespace gl {

constexpr int kNormThreads = 256;

struct NormForward {
  const char *x, *residual, *gamma;
  char *h, *y;
  uint8_t *data, *scale;
  int64_t C;
  float eps;
};

// n consecutive elements of gamma (its own type) as fp32
template <int EL, bool G32>
__device__ __forceinline__ void load_gamma(const char *gamma, int64_t c, float *g) {
  using V = Vec<EL>;
  if constexpr (G32 && EL != EL_F32) {
    Vec<EL_F32>::load(gamma + c * 4, g);
    Vec<EL_F32>::load(gamma + c * 4 + 16, g + 4);
  } else {
    V::load(gamma + c * elem_bytes(EL), g);
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sum over the workgroup in a fixed order; `part` holds one float a wave.
template <int threads>
__device__ __forceinline__ float block_sum(float v, float *part) {
  v = wave_sum(v);
  __syncthreads();  // the last call's values have been read
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < threads / 64; ++w) s += part[w];
  return s;
}

// One workgroup a row, the row read twice (the second time from cache).
template <int EL, bool G32>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_fwd_kernel(const NormForward p) {
  using V = Vec<EL>;
  constexpr int B = elem_bytes(EL);
  __shared__ float part[kNormThreads / 64];
  const int64_t base = (int64_t)blockIdx.x * p.C;
  const auto load = [&](int64_t c, float *s) {
    V::load(p.x + (base + c) * B, s);
    if (p.residual) {
      float r[V::n];
      V::load(p.residual + (base + c) * B, r);
#pragma unroll
      for (int i = 0; i < V::n; ++i) s[i] += r[i];
    }
  };
  float sq = 0.f;
  for (int64_t c = (int64_t)threadIdx.x * V::n; c < p.C; c += kNormThreads * V::n) {
    float s[V::n];
    load(c, s);
#pragma unroll
    for (int i = 0; i < V::n; ++i) sq = fmaf(s[i], s[i], sq);
  }
  const float rstd = 1.f / sqrtf(block_sum<kNormThreads>(sq, part) / (float)p.C + p.eps);
  for (int64_t c = (int64_t)threadIdx.x * V::n; c < p.C; c += kNormThreads * V::n) {
    float s[V::n], g[V::n];
    load(c, s);
    // h may be x or the residual: each element is written by the thread that has just read it
    if (p.h) V::store(p.h + (base + c) * B, s);
    load_gamma<EL, G32>(p.gamma, c, g);
#pragma unroll
    for (int i = 0; i < V::n; ++i) s[i] = s[i] * rstd * g[i];
    if (p.y) V::store(p.y + (base + c) * B, s);
    if (p.data) {
      uint32_t q[V::n / 4];
      const uint8_t byte = quantize_lanes<V::n>(s, q);
#pragma unroll
      for (int i = 0; i < V::n / 4; ++i) ((uint32_t *)(p.data + base + c))[i] = q[i];
      if (c % 32 == 0) p.scale[(base + c) / 32] = byte;
    }
  }
}

struct NormBackward {
  const char *dy, *h, *dh, *gamma;
  char *dx;
  float *part;  // [gridDim.x][C] sums of dy * xh, or null
  int64_t T, C;
  float eps;
};

// Workgroup b takes rows b, b + gridDim.x, ...; each thread adds up dgamma of its own
// columns over those rows, in row order, in the workgroup's row of `part`.
template <int EL, bool G32>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_bwd_kernel(const NormBackward p) {
  using V = Vec<EL>;
  constexpr int B = elem_bytes(EL);
  __shared__ float part[kNormThreads / 64];
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int64_t base = t * p.C;
    float hh = 0.f, vh = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * V::n; c < p.C; c += kNormThreads * V::n) {
      float h[V::n], d[V::n], g[V::n];
      V::load(p.h + (base + c) * B, h);
      V::load(p.dy + (base + c) * B, d);
      load_gamma<EL, G32>(p.gamma, c, g);
#pragma unroll
      for (int i = 0; i < V::n; ++i) {
        hh = fmaf(h[i], h[i], hh);
        vh = fmaf(d[i] * g[i], h[i], vh);
      }
    }
    hh = block_sum<kNormThreads>(hh, part);
    vh = block_sum<kNormThreads>(vh, part);
    const float rstd = 1.f / sqrtf(hh / (float)p.C + p.eps);
    const float c2 = rstd * rstd * (vh / (float)p.C);  // xh * mean(v * xh) = h * c2
    for (int64_t c = (int64_t)threadIdx.x * V::n; c < p.C; c += kNormThreads * V::n) {
      float h[V::n], d[V::n], g[V::n], o[V::n];
      V::load(p.h + (base + c) * B, h);
      V::load(p.dy + (base + c) * B, d);
      load_gamma<EL, G32>(p.gamma, c, g);
#pragma unroll
      for (int i = 0; i < V::n; ++i) o[i] = rstd * (d[i] * g[i] - h[i] * c2);
      if (p.dh) {
        float r[V::n];
        V::load(p.dh + (base + c) * B, r);
#pragma unroll
        for (int i = 0; i < V::n; ++i) o[i] += r[i];
      }
      V::store(p.dx + (base + c) * B, o);
      if (p.part) {
        float *a = p.part + (int64_t)blockIdx.x * p.C + c;
#pragma unroll
        for (int i = 0; i < V::n; ++i) a[i] = (t == blockIdx.x ? 0.f : a[i]) + d[i] * (h[i] * rstd);
      }
    }
  }
}

// dgamma of 64 columns a workgroup: wave w adds up rows w, w + 4, ... of the partial
// sums, then the four sums are added in order.
template <int EL_OUT>
__global__ __launch_bounds__(256) void rmsnorm_dgamma_kernel(const float *__restrict__ part, int rows, int64_t C,
                                                             int accumulate, void *__restrict__ dgamma) {
  __shared__ float sums[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < C)
    for (int r = wave; r < rows; r += 4) s += part[(int64_t)r * C + c];
  sums[wave][lane] = s;
  __syncthreads();
  if (wave || c >= C) return;
  s = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
  if constexpr (EL_OUT == EL_F32) {
    float *o = (float *)dgamma + c;
    *o = accumulate ? *o + s : s;
  } else {
    constexpr bool F16 = EL_OUT == EL_F16;
    uint16_t *o = (uint16_t *)dgamma + c;
    *o = f32_to_h16<F16>(accumulate ? h16_to_f32<F16>(*o) + s : s);
  }
}

template <class F>
static void each_type(int el, bool g32, F f) {
  if (el == EL_F32)
    f(std::integral_constant<int, EL_F32>(), std::true_type());
  else if (el == EL_F16)
    g32 ? f(std::integral_constant<int, EL_F16>(), std::true_type())
        : f(std::integral_constant<int, EL_F16>(), std::false_type());
  else
    g32 ? f(std::integral_constant<int, EL_BF16>(), std::true_type())
        : f(std::integral_constant<int, EL_BF16>(), std::false_type());
}

hipError_t launch_rmsnorm_fwd(int el, bool g32, int64_t T, int64_t C, const void *x, const void *residual,
                              const void *gamma, float eps, void *h, void *y, uint8_t *data, uint8_t *scale,
                              hipStream_t s) {
  const NormForward p{(const char *)x, (const char *)residual, (const char *)gamma, (char *)h, (char *)y,
                      data, scale, C, eps};
  each_type(el, g32, [&](auto e, auto g) {
    hipLaunchKernelGGL((rmsnorm_fwd_kernel<e(), g()>), dim3((unsigned)T), dim3(kNormThreads), 0, s, p);
  });
  return hipGetLastError();
}

// Workgroups of the backward: each leaves one row of partial dgamma sums.
int rmsnorm_bwd_blocks(int64_t T) { return (int)min64(T, 512); }

hipError_t launch_rmsnorm_bwd(int el, bool g32, int64_t T, int64_t C, const void *dy, const void *dh, const void *h,
                              const void *gamma, float eps, void *dx, int el_dgamma, void *dgamma, int accumulate,
                              float *part, hipStream_t s) {
  const int blocks = rmsnorm_bwd_blocks(T);
  const NormBackward p{(const char *)dy, (const char *)h, (const char *)dh, (const char *)gamma, (char *)dx,
                       dgamma ? part : nullptr, T, C, eps};
  if (blocks)
    each_type(el, g32, [&](auto e, auto g) {
      hipLaunchKernelGGL((rmsnorm_bwd_kernel<e(), g()>), dim3(blocks), dim3(kNormThreads), 0, s, p);
    });
  if (dgamma) {
    const dim3 grid((unsigned)((C + 63) / 64));
    if (el_dgamma == EL_F32)
      hipLaunchKernelGGL(rmsnorm_dgamma_kernel<EL_F32>, grid, dim3(256), 0, s, part, blocks, C, accumulate, dgamma);
    else if (el_dgamma == EL_F16)
      hipLaunchKernelGGL(rmsnorm_dgamma_kernel<EL_F16>, grid, dim3(256), 0, s, part, blocks, C, accumulate, dgamma);
    else
      hipLaunchKernelGGL(rmsnorm_dgamma_kernel<EL_BF16>, grid, dim3(256), 0, s, part, blocks, C, accumulate, dgamma);
  }
  return hipGetLastError();
}

}  // namespace gl
