// What the grouped products with a gated or a scaled epilogue share: the activations, the
// arguments of a launch, the element types of the operands with their matrix instruction, the
// lookup of a row tile's group, and the epilogue of four neighbouring output columns of a row.
//
//   h = x W_g^T (times x_scale[row] w_scale[g][col] for 8-bit integers) + b_g
//   plain     y = h
//   gated     W_g has 2 F rows, the gate's first: a = act(h[:, :F]) h[:, F:]
//   gradient  from h and da: dh = [da h_u act'(h_g), da act(h_g)]
//
// Everything from the products' sums on is fp32 (sums of 8-bit codes are exact in int32 and
// rounded once to fp32); every output is rounded once, from the fp32 values.
#pragma once

#include <type_traits>

#include "gl_vec.hpp"

namespace gl {

enum { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

// sigmoid by the hardware's exp2 and reciprocal (each within an ulp of fp32): 4 instructions
// where the correctly rounded division alone takes ten.
__device__ __forceinline__ float sigmoid_fast(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// act(v), and with SLOPE also act'(v).  Infinities get the limits (0 and slope 0, or v and slope 1) and NaN stays NaN:
// beyond +-100 each activation and slope is its limit in fp32, so v is held to that range
// wherever an infinity would meet a zero.
template <bool SLOPE, int ACT>
__device__ __forceinline__ float activate(float v, float &slope) {
  const float lo = v < -100.f ? -100.f : v;  // NaN stays
  const float c = lo > 100.f ? 100.f : lo;
  if constexpr (ACT == ACT_GELU) {
    const float p = 0.5f + 0.5f * erff(c * 0.70710678118654752f);
    if (SLOPE) slope = p + c * 0.3989422804014327f * __builtin_amdgcn_exp2f(c * c * -0.72134752044448170f);
    return lo * p;
  } else if constexpr (ACT == ACT_GELU_TANH) {  // (1 + tanh(z / 2)) / 2 is sigmoid(z)
    const float c2 = c * c;
    const float p = sigmoid_fast(c * (1.5957691216057308f + 0.07135481282651713f * c2));
    if (SLOPE) slope = p + c * p * (1.f - p) * (1.5957691216057308f + 0.21406443847955140f * c2);
    return lo * p;
  } else {
    const float p = sigmoid_fast(c);
    if (SLOPE) slope = p + c * p * (1.f - p);
    return lo * p;
  }
}
// Runs f with the activation as a compile-time tag: one test for many values.
template <class F>
__device__ __forceinline__ void with_activation(int act, F f) {
  if (act == ACT_GELU) f(std::integral_constant<int, ACT_GELU>{});
  else if (act == ACT_GELU_TANH) f(std::integral_constant<int, ACT_GELU_TANH>{});
  else f(std::integral_constant<int, ACT_SILU>{});
}

// ------------------------------------------------------------ operands --
// The operands' element type: bytes and the matrix instruction over 16 bytes of a lane's row.
// Lane l holds bytes of row l % 16 of either operand, the quarters l / 16 of the wave holding
// different contraction values, the same in both; the sum comes as four consecutive rows of
// the first operand, 4 (l / 16) .., of column l % 16, a row of the second.
enum { IN_BF16 = 0, IN_F32 = 1, IN_F16 = 2, IN_I8 = 3 };
constexpr int in_bytes(int in) { return in == IN_F32 ? 4 : in == IN_I8 ? 1 : 2; }

template <int IN>
struct Operand {
  typedef f32x4_t acc_t;
  __device__ static __forceinline__ acc_t mma(i32x4_t a, i32x4_t b, acc_t c) {
    if constexpr (IN == IN_F16) {
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                    0, 0, 0);
    } else if constexpr (IN == IN_BF16) {
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                     c, 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(a[i]), __int_as_float(b[i]), c, 0, 0, 0);
      return c;
    }
  }
};
template <>
struct Operand<IN_I8> {
  typedef i32x4_t acc_t;
  __device__ static __forceinline__ acc_t mma(i32x4_t a, i32x4_t b, acc_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};

// ------------------------------------------------------------- a launch --
enum { EPI_GLU = 0, EPI_GLU_GRAD = 1, EPI_PLAIN = 2 };

struct GluParams {
  const char *x;              // [T, K]
  const char *w;              // [G, N, K] or
  const char *const *w_ptrs;  // G x [N, K]; N = 2 F, plain: F
  const void *bias;           // [G, N] of the output's type
  const void *const *bias_ptrs;
  const float *x_scale;  // 8-bit integers: [T]
  const float *w_scale;  // and [G, N] or
  const float *const *w_scale_ptrs;
  void *out;       // [T, F] a or y; gradient: dh [T, 2 F]
  void *h;         // forward: [T, 2 F] or null
  const void *da;  // gradient: [T, F]
  void *a;         // gradient: [T, F] or null
  const void *ws;
  int G, act;
  int64_t T, K, F;
};

template <int IN, int EPI>
__device__ __forceinline__ const char *group_weights(const GluParams &p, int g) {
  const int64_t n = EPI == EPI_PLAIN ? p.F : 2 * p.F;
  return p.w ? p.w + (int64_t)g * n * p.K * in_bytes(IN) : p.w_ptrs[g];
}

// Four consecutive elements of a tensor as fp32 values, and back (16-bit types: 8 bytes).
template <int EL>
__device__ __forceinline__ float4 load4(const void *base, int64_t at) {
  if constexpr (EL == EL_F32) {
    return *(const float4 *)((const float *)base + at);
  } else {
    const uint2 u = *(const uint2 *)((const uint16_t *)base + at);
    constexpr bool H = EL == EL_F16;
    return make_float4(h16_to_f32<H>(u.x & 0xffff), h16_to_f32<H>(u.x >> 16), h16_to_f32<H>(u.y & 0xffff),
                       h16_to_f32<H>(u.y >> 16));
  }
}
template <int EL>
__device__ __forceinline__ void put4(void *base, int64_t at, float4 v) {
  if constexpr (EL == EL_F32)
    *(float4 *)((float *)base + at) = v;
  else
    *(uint2 *)((uint16_t *)base + at) =
        make_uint2(pack_h16x2<EL == EL_F16>(v.x, v.y), pack_h16x2<EL == EL_F16>(v.z, v.w));
}

// What four columns of a group add to a row's sums: the bias, and for 8-bit integers the
// channels' scales.
struct ColumnTerms {
  float4 scale, bias;
};
template <int IN, int EL, int EPI>
__device__ __forceinline__ ColumnTerms column_terms(const GluParams &p, int g, int64_t col) {
  const int64_t n = EPI == EPI_PLAIN ? p.F : 2 * p.F;
  ColumnTerms c;
  c.scale = c.bias = make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (IN == IN_I8) {
    const float *s = p.w_scale ? p.w_scale + (int64_t)g * n : p.w_scale_ptrs[g];
    c.scale = make_float4(s[col], s[col + 1], s[col + 2], s[col + 3]);  // a group's scales may sit at any word
  }
  if (p.bias)
    c.bias = load4<EL>(p.bias, (int64_t)g * n + col);
  else if (p.bias_ptrs)
    c.bias = load4<EL>(p.bias_ptrs[g], col);
  return c;
}

template <int IN>
__device__ __forceinline__ float4 finish(typename Operand<IN>::acc_t s, float row_scale, const ColumnTerms &c) {
  if constexpr (IN == IN_I8)
    return make_float4((float)s[0] * (row_scale * c.scale.x) + c.bias.x,
                       (float)s[1] * (row_scale * c.scale.y) + c.bias.y,
                       (float)s[2] * (row_scale * c.scale.z) + c.bias.z,
                       (float)s[3] * (row_scale * c.scale.w) + c.bias.w);
  else
    return make_float4(s[0] + c.bias.x, s[1] + c.bias.y, s[2] + c.bias.z, s[3] + c.bias.w);
}

template <bool SLOPE, int ACT>
__device__ __forceinline__ float4 activate4(float4 v, float4 &slope) {
  float4 o;
  o.x = activate<SLOPE, ACT>(v.x, slope.x);
  o.y = activate<SLOPE, ACT>(v.y, slope.y);
  o.z = activate<SLOPE, ACT>(v.z, slope.z);
  o.w = activate<SLOPE, ACT>(v.w, slope.w);
  return o;
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}

// The gated epilogues for columns col .. col + 3 of row `row`: g and u are the finished
// values of h's two halves there.
template <int EL, int EPI, int ACT>
__device__ __forceinline__ void gated4(const GluParams &p, int64_t row, int64_t col, float4 g, float4 u) {
  float4 slope = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 y = activate4<EPI == EPI_GLU_GRAD, ACT>(g, slope);
  if constexpr (EPI == EPI_GLU) {
    put4<EL>(p.out, row * p.F + col, mul4(y, u));
    if (p.h) {
      put4<EL>(p.h, row * 2 * p.F + col, g);
      put4<EL>(p.h, row * 2 * p.F + p.F + col, u);
    }
  } else {
    const float4 d = load4<EL>(p.da, row * p.F + col);
    put4<EL>(p.out, row * 2 * p.F + col, mul4(mul4(d, u), slope));
    put4<EL>(p.out, row * 2 * p.F + p.F + col, mul4(d, y));
    if (p.a) put4<EL>(p.a, row * p.F + col, mul4(y, u));
  }
}

}  // namespace gl
