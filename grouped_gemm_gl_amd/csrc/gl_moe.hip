// The expert layer for a few tokens: for token t with experts e_j = ids[t, j] and
// weights w_j
//   y_t = residual_t + sum_j w_j (W2_e SwiGLU(W1_e x_t + b1_e) + b2_e)
// in two kernels, without sorting or gathering rows.  A slot whose id is no expert of
// this call, or whose weight is 0, takes no part.
//
// The first kernel leaves a = SwiGLU(W1 x + b1) of every slot in the workspace in fp32,
// the second contracts it with W2 and adds up a token's slots.
#include <type_traits>

#include "gl_vec.hpp"

namespace gl {

constexpr int kMoeThreads = 256, kMoeWaves = kMoeThreads / 64;
enum { EL_MX = 3 };  // weights: E4M3 codes with an E8M0 scale per 32 of a row

struct MoeWeight {
  const char *w;
  const char *const *w_ptrs;
  const uint8_t *scale;
  const uint8_t *const *scale_ptrs;
  const char *bias;
  const char *const *bias_ptrs;
  int64_t rows, cols;  // of one expert's matrix
};

struct MoeParams {
  const char *x;
  const int32_t *ids;
  const float *gates;
  MoeWeight w1, w2;
  const char *residual;
  char *y;
  float *a;  // [T k][F]
  int T, k, E;
  int64_t K, F, N;
};

__device__ __forceinline__ float e8m0(uint8_t s) {
  return __uint_as_float(s == 0xff ? 0x7fc00000u : s ? (uint32_t)s << 23 : 0x00400000u);
}

// Dot product of row r of expert e's matrix with the fp32 values `in(c, n)` gives, over
// the wave's lanes (the sum is in every lane).
template <int EL, class In>
__device__ __forceinline__ float row_dot(const MoeWeight &m, int e, int64_t r, In in) {
  constexpr int n = EL == EL_F32 ? 4 : 8;
  const int lane = threadIdx.x & 63;
  float s = 0.f;
  if constexpr (EL == EL_MX) {
    const char *w = (m.w_ptrs ? m.w_ptrs[e] : m.w + (int64_t)e * m.rows * m.cols) + r * m.cols;
    const uint8_t *sc = (m.scale_ptrs ? m.scale_ptrs[e] : m.scale + (int64_t)e * m.rows * (m.cols / 32)) +
                        r * (m.cols / 32);
    for (int64_t c = lane * n; c < m.cols; c += 64 * n) {
      const uint2 q = *(const uint2 *)(w + c);
      const float f = e8m0(sc[c / 32]);
      float v[8];
      in(c, v);
      const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true);
      const auto d = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false), g = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true);
      s = fmaf(a[0] * f, v[0], s); s = fmaf(a[1] * f, v[1], s);
      s = fmaf(b[0] * f, v[2], s); s = fmaf(b[1] * f, v[3], s);
      s = fmaf(d[0] * f, v[4], s); s = fmaf(d[1] * f, v[5], s);
      s = fmaf(g[0] * f, v[6], s); s = fmaf(g[1] * f, v[7], s);
    }
  } else {
    constexpr int B = elem_bytes(EL);
    const char *w = (m.w_ptrs ? m.w_ptrs[e] : m.w + (int64_t)e * m.rows * m.cols * B) + r * m.cols * B;
    for (int64_t c = lane * n; c < m.cols; c += 64 * n) {
      float u[n], v[n];
      Vec<EL>::load(w + c * B, u);
      in(c, v);
#pragma unroll
      for (int i = 0; i < n; ++i) s = fmaf(u[i], v[i], s);
    }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  return s;
}

template <int EL>
__device__ __forceinline__ float load_one(const char *p, int64_t i) {
  if constexpr (EL == EL_F32) return ((const float *)p)[i];
  else return h16_to_f32<EL == EL_F16>(((const uint16_t *)p)[i]);
}

template <int EL>
__device__ __forceinline__ float bias_at(const MoeWeight &m, int e, int64_t r) {
  constexpr int B = elem_bytes(EL);
  const char *b = m.bias_ptrs ? m.bias_ptrs[e] : m.bias ? m.bias + (int64_t)e * m.rows * B : nullptr;
  return b ? load_one<EL>(b, r) : 0.f;
}

// Workgroup (slot, 16 columns of a), a wave a column at a time.
template <int EL, int WEL>
__global__ __launch_bounds__(kMoeThreads) void moe_up_kernel(const MoeParams p) {
  const int s = blockIdx.y, t = s / p.k;
  const int e = p.ids[s];
  if (e < 0 || e >= p.E || p.gates[s] == 0.f) return;
  for (int i = threadIdx.x >> 6; i < 16; i += kMoeWaves) {
    const int64_t f = (int64_t)blockIdx.x * 16 + i;
    if (f >= p.F) break;
    const auto in = [&](int64_t c, float *v) {
      Vec<EL>::load(p.x + (t * p.K + c) * elem_bytes(EL), v);
    };
    const float g = row_dot<WEL>(p.w1, e, f, in) + bias_at<EL>(p.w1, e, f);
    const float u = row_dot<WEL>(p.w1, e, p.F + f, in) + bias_at<EL>(p.w1, e, p.F + f);
    if ((threadIdx.x & 63) == 0) p.a[s * p.F + f] = g * sigmoid(g) * u;
  }
}

// Workgroup (token, 16 columns of y).
template <int EL, int WEL>
__global__ __launch_bounds__(kMoeThreads) void moe_down_kernel(const MoeParams p) {
  const int t = blockIdx.y;
  for (int i = threadIdx.x >> 6; i < 16; i += kMoeWaves) {
    const int64_t n = (int64_t)blockIdx.x * 16 + i;
    if (n >= p.N) break;
    float y = p.residual ? load_one<EL>(p.residual, t * p.N + n) : 0.f;
    for (int j = 0; j < p.k; ++j) {
      const int s = t * p.k + j, e = p.ids[s];
      const float w = p.gates[s];
      if (e < 0 || e >= p.E || w == 0.f) continue;
      const auto in = [&](int64_t c, float *v) {
        Vec<EL_F32>::load(p.a + s * p.F + c, v);
        if constexpr (WEL != EL_F32) Vec<EL_F32>::load(p.a + s * p.F + c + 4, v + 4);
      };
      y = fmaf(w, row_dot<WEL>(p.w2, e, n, in) + bias_at<EL>(p.w2, e, n), y);
    }
    if ((threadIdx.x & 63) == 0) {
      if constexpr (EL == EL_F32) ((float *)p.y)[t * p.N + n] = y;
      else ((uint16_t *)p.y)[t * p.N + n] = f32_to_h16<EL == EL_F16>(y);
    }
  }
}

size_t moe_workspace_bytes(int64_t T, int k, int, int64_t F) { return (size_t)T * k * F * 4; }

hipError_t launch_moe(int el, bool mx, int E, int64_t K, int64_t F, int64_t N, int64_t T, int k, const void *x,
                      const int32_t *ids, const float *gates, const void *w1, const void *const *w1_ptrs,
                      const uint8_t *w1_scale, const uint8_t *const *w1_scale_ptrs, const void *b1,
                      const void *const *b1_ptrs, const void *w2, const void *const *w2_ptrs,
                      const uint8_t *w2_scale, const uint8_t *const *w2_scale_ptrs, const void *b2,
                      const void *const *b2_ptrs, const void *residual, void *y, void *ws, hipStream_t s) {
  MoeParams p;
  p.x = (const char *)x;
  p.ids = ids;
  p.gates = gates;
  p.w1 = {(const char *)w1, (const char *const *)w1_ptrs, w1_scale, w1_scale_ptrs, (const char *)b1,
          (const char *const *)b1_ptrs, 2 * F, K};
  p.w2 = {(const char *)w2, (const char *const *)w2_ptrs, w2_scale, w2_scale_ptrs, (const char *)b2,
          (const char *const *)b2_ptrs, N, F};
  p.residual = (const char *)residual;
  p.y = (char *)y;
  p.a = (float *)ws;
  p.T = (int)T;
  p.k = k;
  p.E = E;
  p.K = K;
  p.F = F;
  p.N = N;
  const auto go = [&](auto el_, auto wel) {
    hipLaunchKernelGGL((moe_up_kernel<el_(), wel()>), dim3((unsigned)((F + 15) / 16), (unsigned)(T * k)),
                       dim3(kMoeThreads), 0, s, p);
    hipLaunchKernelGGL((moe_down_kernel<el_(), wel()>), dim3((unsigned)((N + 15) / 16), (unsigned)T),
                       dim3(kMoeThreads), 0, s, p);
  };
  using B = std::integral_constant<int, EL_BF16>;
  using H = std::integral_constant<int, EL_F16>;
  using S = std::integral_constant<int, EL_F32>;
  using M = std::integral_constant<int, EL_MX>;
  if (mx) go(B(), M());
  else if (el == EL_F32) go(S(), S());
  else if (el == EL_F16) go(H(), H());
  else go(B(), B());
  return hipGetLastError();
}

}  // namespace gl
