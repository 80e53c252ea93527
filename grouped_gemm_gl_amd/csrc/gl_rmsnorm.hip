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
//
// Bound by HBM: a row is held in registers between its sum and its output, so every value
// is read once and written once.  16384 rows of 4096 bf16: forward with residual, h, y and
// codes (606 MB) 102 us, 5.9 TB/s; backward with dh and dgamma (537 MB) 109 us for dx and the
// partial sums of dgamma and 5 us for their addition, 4.7 TB/s.  (A copy of 2 GiB reaches
// 4.9 TB/s, reads and writes counted.)
#include <type_traits>

#include "gl_mx.hpp"
#include "gl_vec.hpp"

namespace gl {

constexpr int kNormThreads = 256, kDgThreads = 1024;

struct NormForward {
  const char *x, *residual, *gamma;
  char *h, *y;
  uint8_t *data, *scale;
  int64_t T, C;
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

// Two sums at once; `part` holds two floats a wave.
template <int threads>
__device__ __forceinline__ void block_sum2(float &a, float &b, float *part) {
  a = wave_sum(a);
  b = wave_sum(b);
  __syncthreads();  // the last call's values have been read
  if ((threadIdx.x & 63) == 0) {
    part[2 * (threadIdx.x >> 6)] = a;
    part[2 * (threadIdx.x >> 6) + 1] = b;
  }
  __syncthreads();
  a = b = 0.f;
#pragma unroll
  for (int w = 0; w < threads / 64; ++w) {
    a += part[2 * w];
    b += part[2 * w + 1];
  }
}

// The codes of n values at column c of a row that starts at element `base`.
template <int n>
__device__ __forceinline__ void write_codes(const NormForward &p, int64_t base, int64_t c, const float *y) {
  uint32_t q[n / 4];
  const uint8_t byte = quantize_lanes<n>(y, q);
  if constexpr (n == 8) *(uint2 *)(p.data + base + c) = make_uint2(q[0], q[1]);
  else *(uint32_t *)(p.data + base + c) = q[0];
  if (c % 32 == 0) p.scale[(base + c) / 32] = byte;
}

// Threads that share a row (a wave or a whole workgroup) and the rows of a workgroup.
// Each thread holds VPT 16-byte vectors of its row in registers, so a row of up to
// threads * VPT vectors is read once.
template <int NT>
struct RowSplit {
  static constexpr int threads = NT < kNormThreads ? kNormThreads : NT;
  static constexpr int rows = threads / NT;
};

// Sum over the NT threads of a row.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float *part) {
  if constexpr (NT == 64) return wave_sum(v);
  else return block_sum<NT>(v, part);
}

template <int EL, bool G32, int NT, int VPT>
__global__ __launch_bounds__(RowSplit<NT>::threads) void rmsnorm_fwd_kernel(const NormForward p) {
  using V = Vec<EL>;
  constexpr int B = elem_bytes(EL);
  __shared__ float part[NT / 64];
  const int64_t t = (int64_t)blockIdx.x * RowSplit<NT>::rows + threadIdx.x / NT;
  if (t >= p.T) return;  // (rows of a wave: no barrier follows)
  const int64_t base = t * p.C;
  const int c0 = (threadIdx.x % NT) * V::n;
  float s[VPT][V::n];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = c0 + i * NT * V::n;
#pragma unroll
    for (int k = 0; k < V::n; ++k) s[i][k] = 0.f;
    if (c < p.C) V::load(p.x + (base + c) * B, s[i]);
  }
  if (p.residual)
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = c0 + i * NT * V::n;
      if (c < p.C) {
        float r[V::n];
        V::load(p.residual + (base + c) * B, r);
#pragma unroll
        for (int k = 0; k < V::n; ++k) s[i][k] += r[k];
      }
    }
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < V::n; ++k) sq = fmaf(s[i][k], s[i][k], sq);
  const float rstd = 1.f / sqrtf(row_sum<NT>(sq, part) / (float)p.C + p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = c0 + i * NT * V::n;
    if (c >= p.C) break;
    if (p.h) V::store(p.h + (base + c) * B, s[i]);
    float g[V::n];
    load_gamma<EL, G32>(p.gamma, c, g);
#pragma unroll
    for (int k = 0; k < V::n; ++k) s[i][k] = s[i][k] * rstd * g[k];
    if (p.y) V::store(p.y + (base + c) * B, s[i]);
    if (p.data) write_codes<V::n>(p, base, c, s[i]);
  }
}

// Rows past what registers hold: one workgroup a row, the row read twice.
template <int EL, bool G32>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_fwd_long_kernel(const NormForward p) {
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
    if (p.data) write_codes<V::n>(p, base, c, s);
  }
}

struct NormBackward {
  const char *dy, *h, *dh, *gamma;
  char *dx;
  float *part;  // [gridDim.x][C] sums of dy * xh, or null
  int64_t T, C;
  float eps;
};

// Workgroup b takes rows b, b + gridDim.x, ... (RowSplit<NT>::rows at a time); each thread
// adds up dgamma of its own columns over those rows, in row order, in registers.  The next
// row's h and dy are on their way while this one is reduced.
template <int EL, bool G32, int NT, int VPT>
__global__ __launch_bounds__(RowSplit<NT>::threads) void rmsnorm_bwd_kernel(const NormBackward p) {
  using V = Vec<EL>;
  constexpr int B = elem_bytes(EL), R = RowSplit<NT>::rows;
  __shared__ float part[2 * (NT / 64)];
  __shared__ float rows[R > 1 ? R * NT * VPT * V::n : 1];
  const int tid = threadIdx.x % NT, sub = threadIdx.x / NT, c0 = tid * V::n;
  float dg[VPT][V::n];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < V::n; ++k) dg[i][k] = 0.f;
  uint4 h[VPT], d[VPT];
  const auto load = [&](int64_t t, uint4 *h, uint4 *d) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = c0 + i * NT * V::n;
      h[i] = d[i] = make_uint4(0, 0, 0, 0);
      if (t < p.T && c < p.C) {
        h[i] = *(const uint4 *)(p.h + (t * p.C + c) * B);
        d[i] = *(const uint4 *)(p.dy + (t * p.C + c) * B);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t t = (int64_t)blockIdx.x * R + sub;
  load(t, h, d);
  for (; t < p.T; t += step) {
    uint4 nh[VPT], nd[VPT], r[VPT];
    if (p.dh)
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (c0 + i * NT * V::n < p.C) r[i] = *(const uint4 *)(p.dh + (t * p.C + c0 + i * NT * V::n) * B);
    load(t + step, nh, nd);
    float hh = 0.f, vh = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = c0 + i * NT * V::n;
      if (c >= p.C) break;
      float hf[V::n], df[V::n], g[V::n];
      V::load(&h[i], hf);
      V::load(&d[i], df);
      load_gamma<EL, G32>(p.gamma, c, g);
#pragma unroll
      for (int k = 0; k < V::n; ++k) {
        hh = fmaf(hf[k], hf[k], hh);
        vh = fmaf(df[k] * g[k], hf[k], vh);
      }
    }
    if constexpr (NT == 64) {
      hh = wave_sum(hh);
      vh = wave_sum(vh);
    } else {
      block_sum2<NT>(hh, vh, part);
    }
    const float rstd = 1.f / sqrtf(hh / (float)p.C + p.eps);
    const float c2 = rstd * rstd * (vh / (float)p.C);  // xh * mean(v * xh) = h * c2
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = c0 + i * NT * V::n;
      if (c >= p.C) break;
      float hf[V::n], df[V::n], g[V::n], o[V::n];
      V::load(&h[i], hf);
      V::load(&d[i], df);
      load_gamma<EL, G32>(p.gamma, c, g);
#pragma unroll
      for (int k = 0; k < V::n; ++k) {
        o[k] = rstd * (df[k] * g[k] - hf[k] * c2);
        dg[i][k] += df[k] * (hf[k] * rstd);
      }
      if (p.dh) {
        float rf[V::n];
        V::load(&r[i], rf);
#pragma unroll
        for (int k = 0; k < V::n; ++k) o[k] += rf[k];
      }
      V::store(p.dx + (t * p.C + c) * B, o);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      h[i] = nh[i];
      d[i] = nd[i];
    }
  }
  if (!p.part) return;
  if constexpr (R > 1) {  // the workgroup's rows add up in order
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < V::n; ++k) rows[(sub * VPT + i) * NT * V::n + c0 + k] = dg[i][k];
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < V::n; ++k)
#pragma unroll
        for (int r = 1; r < R; ++r) dg[i][k] += rows[(r * VPT + i) * NT * V::n + c0 + k];
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = c0 + i * NT * V::n;
    if (c >= p.C) break;
    float *o = p.part + (int64_t)blockIdx.x * p.C + c;
#pragma unroll
    for (int k = 0; k < V::n; k += 4) *(float4 *)(o + k) = make_float4(dg[i][k], dg[i][k + 1], dg[i][k + 2], dg[i][k + 3]);
  }
}

// Rows past what registers hold: dgamma is added up in the workgroup's row of `part`.
template <int EL, bool G32>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_bwd_long_kernel(const NormBackward p) {
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

// dgamma of 64 columns a workgroup: each of 16 waves adds up every 16th of the partial
// rows, then the waves' sums are added in order.
template <int EL_OUT>
__global__ __launch_bounds__(kDgThreads) void rmsnorm_dgamma_kernel(const float *__restrict__ part, int rows, int64_t C,
                                                                    int accumulate, void *__restrict__ dgamma) {
  constexpr int kWaves = kDgThreads / 64;
  __shared__ float sums[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < C)
#pragma unroll 8
    for (int r = wave; r < rows; r += kWaves) s += part[(int64_t)r * C + c];
  sums[wave][lane] = s;
  __syncthreads();
  if (wave || c >= C) return;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += sums[w][lane];
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

// How a row's 16-byte vectors are held in registers: f(threads, vectors a thread), or
// too_long() past 2048 vectors.  The forward does best with few vectors a thread (one row of
// 4096 bf16 over 512 threads 106 us, over 256 threads 114 us, at 16384 rows); the backward,
// which keeps a row ahead in flight and its dgamma sums, with two (102 and 107 us).
template <bool kForward, class F, class L>
static void each_split(int64_t vectors, F f, L too_long) {
  using std::integral_constant;
  using One = integral_constant<int, 1>;
  using Two = integral_constant<int, 2>;
  if (vectors <= 64) f(integral_constant<int, 64>(), One());
  else if (vectors <= 128) f(integral_constant<int, 64>(), Two());
  else if (vectors <= 256) f(integral_constant<int, 256>(), One());
  else if (vectors <= 512) f(integral_constant<int, kForward ? 512 : 256>(), integral_constant<int, kForward ? 1 : 2>());
  else if (vectors <= 1024) f(integral_constant<int, 512>(), Two());
  else if (vectors <= 2048) f(integral_constant<int, 1024>(), Two());
  else too_long();
}

hipError_t launch_rmsnorm_fwd(int el, bool g32, int64_t T, int64_t C, const void *x, const void *residual,
                              const void *gamma, float eps, void *h, void *y, uint8_t *data, uint8_t *scale,
                              hipStream_t s) {
  // f(a slice of the rows, its workgroups)
  const auto slices = [&](int threads, int rows, auto f) {
    const int64_t step = kSliceThreads / threads * rows, row = C * elem_bytes(el);
    const auto at = [](auto *q, int64_t bytes) { return q ? q + bytes : nullptr; };
    for (int64_t t = 0; t < T; t += step) {
      const int64_t n = min64(T - t, step);
      f(NormForward{(const char *)x + t * row, at((const char *)residual, t * row), (const char *)gamma,
                    at((char *)h, t * row), at((char *)y, t * row), at(data, t * C), at(scale, t * (C / 32)), n, C, eps},
        dim3((unsigned)((n + rows - 1) / rows)));
    }
  };
  each_type(el, g32, [&](auto e, auto g) {
    each_split<true>(
        C / Vec<e()>::n,
        [&](auto nt, auto vpt) {
          using S = RowSplit<nt()>;
          slices(S::threads, S::rows, [&](const NormForward &p, dim3 grid) {
            hipLaunchKernelGGL((rmsnorm_fwd_kernel<e(), g(), nt(), vpt()>), grid, dim3(S::threads), 0, s, p);
          });
        },
        [&] {
          slices(kNormThreads, 1, [&](const NormForward &p, dim3 grid) {
            hipLaunchKernelGGL((rmsnorm_fwd_long_kernel<e(), g()>), grid, dim3(kNormThreads), 0, s, p);
          });
        });
  });
  return hipGetLastError();
}

// Workgroups of the backward; each leaves one row of partial dgamma sums, so few rows get
// one a CU, and short rows, whose workgroups hold less in flight, more of them.
int rmsnorm_bwd_blocks(int64_t T, int64_t C) {
  return T < 1024 ? (int)min64(T, 256) : C <= 2048 ? 1024 : 512;
}

hipError_t launch_rmsnorm_bwd(int el, bool g32, int64_t T, int64_t C, const void *dy, const void *dh, const void *h,
                              const void *gamma, float eps, void *dx, int el_dgamma, void *dgamma, int accumulate,
                              float *part, hipStream_t s) {
  const int blocks = rmsnorm_bwd_blocks(T, C);
  const NormBackward p{(const char *)dy, (const char *)h, (const char *)dh, (const char *)gamma, (char *)dx,
                       dgamma ? part : nullptr, T, C, eps};
  if (blocks)
    each_type(el, g32, [&](auto e, auto g) {
      each_split<false>(
          C / Vec<e()>::n,
          [&](auto nt, auto vpt) {
            hipLaunchKernelGGL((rmsnorm_bwd_kernel<e(), g(), nt(), vpt()>), dim3(blocks),
                               dim3(RowSplit<nt()>::threads), 0, s, p);
          },
          [&] { hipLaunchKernelGGL((rmsnorm_bwd_long_kernel<e(), g()>), dim3(blocks), dim3(kNormThreads), 0, s, p); });
    });
  if (dgamma) {
    const dim3 grid((unsigned)((C + 63) / 64));
    if (el_dgamma == EL_F32)
      hipLaunchKernelGGL(rmsnorm_dgamma_kernel<EL_F32>, grid, dim3(kDgThreads), 0, s, part, blocks, C, accumulate, dgamma);
    else if (el_dgamma == EL_F16)
      hipLaunchKernelGGL(rmsnorm_dgamma_kernel<EL_F16>, grid, dim3(kDgThreads), 0, s, part, blocks, C, accumulate, dgamma);
    else
      hipLaunchKernelGGL(rmsnorm_dgamma_kernel<EL_BF16>, grid, dim3(kDgThreads), 0, s, part, blocks, C, accumulate, dgamma);
  }
  return hipGetLastError();
}

}  // namespace gl
