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

#include "gl_gemm_tile.hpp"
#include "gl_glu_choice.hpp"
#include "gl_vec.hpp"

namespace gl {

enum { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

// sigmoid by the hardware's exp2 and reciprocal (each within an ulp of fp32): 4 instructions
// where the correctly rounded division alone takes ten.
__device__ __forceinline__ float sigmoid_fast(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// Phi(v), the normal distribution, given e = exp(-v^2 / 2): for v < 0 it is e t P(t) with
// t = 1 / (1 + 0.35 |v|), and 1 - Phi(-v) for the others.  P, of degree 8, is the least relative error's
// for v down to -13.5, where e leaves fp32 (3e-8; in fp32 arithmetic 3e-7 without e's own).  0.5 + 0.5
// erf(v / sqrt 2) cancels where v is negative: 4% off at -5, 0 from -5.6 on.
__device__ __forceinline__ float normal_cdf(float v, float e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(v), 0.35f, 1.f));
  float p = -0.02912587672472f;
  p = fmaf(p, t, 0.143872290849686f);
  p = fmaf(p, t, -0.255504667758942f);
  p = fmaf(p, t, 0.158929407596588f);
  p = fmaf(p, t, -0.0229372195899487f);
  p = fmaf(p, t, 0.105432972311974f);
  p = fmaf(p, t, 0.119852431118488f);
  p = fmaf(p, t, 0.139859080314636f);
  p = fmaf(p, t, 0.139621570706368f);
  const float q = p * t * e;
  return v < 0.f ? q : 1.f - q;
}

// act(v) = v p, and with SLOPE act'(v) = p + v p'.  Infinities get the limits (0 and slope 0, or
// v and slope 1) and NaN stays NaN: where p or p' is 0 in fp32, so is its product with v, an
// infinite v's too.
template <bool SLOPE, int ACT>
__device__ __forceinline__ float activate(float v, float &slope) {
  auto times = [](float v, float p) { return p == 0.f ? 0.f : v * p; };
  if constexpr (ACT == ACT_GELU) {
    const float e = __builtin_amdgcn_exp2f(v * v * -0.72134752044448170f);  // exp(-v^2 / 2)
    const float p = normal_cdf(v, e);
    if (SLOPE) slope = p + times(v, 0.3989422804014327f * e);
    return times(v, p);
  } else if constexpr (ACT == ACT_GELU_TANH) {  // (1 + tanh(z / 2)) / 2 is sigmoid(z)
    // each step with one literal: two would hold a register each
    const float v3 = v * v * v;
    const float p = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(fmaf(v, -2.3022081983f, v3 * -0.1029432397f)));
    if (SLOPE) {
      const float q = p * (1.f - p);
      slope = p + (q == 0.f ? 0.f : q * fmaf(v, 1.5957691216f, v3 * 0.2140644385f));
    }
    return times(v, p);
  } else {
    const float p = sigmoid_fast(v);
    if (SLOPE) slope = p + times(v, p * (1.f - p));
    return times(v, p);
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
// (IN_BF16 .. IN_I8: gl_glu_choice.hpp)

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

// A long contraction in fp32: what the matrix instruction added up over `every` steps joins the sum of
// those before, so that no chain of additions is longer than kFp32Chain values and the number of chunks.
// Error of the norm against 64 bits, one chain / chunks of 512 / of 256: dx of 5 groups, 221 rows, K 7040, 2F
// 12080 2.0e-6 / 4.1e-7 / 3.2e-7; of 2F 2048 5.7e-7 / 4.1e-7 / 2.9e-7, and a library product, which cuts some of its
// contractions, 2.0e-6 and 4.1e-7.  Time: 1332 / 1357 / 1361 us and 57.3 / 57.8 / 57.9.  Nothing for the
// other types, whose outputs are rounded to 16 bits or whose sums are exact, nor on tiles of 256 rows, whose
// accumulators fill the registers: there a chain is the contraction, as in the library's products.
constexpr int kFp32Chain = 256;
template <int IN, int N>
struct ChunkSums {
  __device__ __forceinline__ ChunkSums() {}
  __device__ __forceinline__ void step(int, int, typename Operand<IN>::acc_t *) {}
  __device__ __forceinline__ void end(typename Operand<IN>::acc_t *) {}
};
template <int N>
struct ChunkSums<IN_F32, N> {
  f32x4_t before[N];
  __device__ __forceinline__ ChunkSums() {
#pragma unroll
    for (int i = 0; i < N; ++i) before[i] = f32x4_t{0, 0, 0, 0};
  }
  // after step s (the same in every lane), `every` a power of two
  __device__ __forceinline__ void step(int s, int every, f32x4_t *acc) {
    if ((s & (every - 1)) != every - 1) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      before[i] += acc[i];
      acc[i] = f32x4_t{0, 0, 0, 0};
    }
  }
  __device__ __forceinline__ void end(f32x4_t *acc) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += before[i];
  }
};

// ------------------------------------------------------------- a launch --
enum { EPI_GLU = 0, EPI_GLU_GRAD = 1, EPI_PLAIN = 2, EPI_DX = 3, EPI_DW = 4 };

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
  // The backward's products on the same tiles.  dx [T, F] = x [T, K] w [G, K, F], x being the
  // gradient of h; dW [G, N, F] = x^T w for each group's rows of x [T, N] and w [T, F].
  void *const *out_ptrs;  // dW: G x [N, F], or out
  int64_t N;
  int accumulate;
};

// The products of the backward, out = dh w (dx) or dh^T x (dW), for each group.
struct BackParams {
  const char *a;  // dh [T, 2F]
  const char *b;  // dx: w [G, 2F, K] or
  const char *const *b_ptrs;
  const char *x;  // dW: x [T, K]
  void *out;      // dx [T, K]; dW [G, 2F, K] or
  void *const *out_ptrs;
  const void *ws;
  int G, accumulate;
  int64_t T, K, N;  // N = 2F
};

// The row tiles of a launch and their groups.  Below 64 groups the wave's lanes hold the whole tables
// (lane i: group i), so that a workgroup's first loads wait for one round trip to memory where the
// tables one after the other take four.
struct RowTiles {
  const int64_t *__restrict__ off;
  const int32_t *__restrict__ pre;
  int G, pre_l = 0;
  int64_t off_l = 0;
  bool held;
  __device__ __forceinline__ RowTiles(const WsView &ws, int G, int rows)
      : off(ws.off), pre(ws.pre[tile_rows_index(rows)]), G(G), held(G < 64) {
    if (held) {
      const int i = min((int)(threadIdx.x & 63), G);
      pre_l = pre[i];
      off_l = off[i];
    }
  }
  // (read back as uniform: a buffer resource's length from them is otherwise taken as the lanes' own,
  // and every load goes through a loop over its values)
  __device__ __forceinline__ int tile(int g) const {
    return held ? __builtin_amdgcn_readlane(pre_l, g) : __builtin_amdgcn_readfirstlane(pre[g]);
  }
  __device__ __forceinline__ int64_t row(int g) const {
    if (!held) return (int64_t)(uintptr_t)gemm::uniform_ptr((const char *)(uintptr_t)off[g]);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)off_l, g);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)off_l >> 32), g);
    return (int64_t)(((uint64_t)hi << 32) | lo);
  }
  // the group of row tile q (the last whose first tile is not after q)
  __device__ __forceinline__ int group(int q) const {
    if (!held) return __builtin_amdgcn_readfirstlane(find_group(pre, G, q));
    return __popcll(__ballot((int)(threadIdx.x & 63) <= G && pre_l <= q)) - 1;
  }
};

template <int IN, int EPI>
__device__ __forceinline__ const char *group_weights(const GluParams &p, int g) {
  const int64_t n = EPI == EPI_GLU || EPI == EPI_GLU_GRAD ? 2 * p.F : p.F;
  return p.w ? p.w + (int64_t)g * n * p.K * in_bytes(IN) : p.w_ptrs[g];
}

// Four consecutive elements of a tensor, as they are and as fp32 values (16-bit types: 8 bytes).
template <int EL>
struct Quad {
  typedef uint2 raw;
  __device__ static __forceinline__ float4 value(uint2 u) {
    constexpr bool H = EL == EL_F16;
    return make_float4(h16_to_f32<H>(u.x & 0xffff), h16_to_f32<H>(u.x >> 16), h16_to_f32<H>(u.y & 0xffff),
                       h16_to_f32<H>(u.y >> 16));
  }
  __device__ static __forceinline__ uint2 pack(float4 v) {
    return make_uint2(pack_h16x2<EL == EL_F16>(v.x, v.y), pack_h16x2<EL == EL_F16>(v.z, v.w));
  }
};
template <>
struct Quad<EL_F32> {
  typedef float4 raw;
  __device__ static __forceinline__ float4 value(float4 v) { return v; }
  __device__ static __forceinline__ float4 pack(float4 v) { return v; }
};
template <int EL>
__device__ __forceinline__ typename Quad<EL>::raw load_raw4(const void *base, int64_t at) {
  return *(const typename Quad<EL>::raw *)((const char *)base + at * elem_bytes(EL));
}
template <int EL>
__device__ __forceinline__ float4 load4(const void *base, int64_t at) {
  return Quad<EL>::value(load_raw4<EL>(base, at));
}
template <int EL>
__device__ __forceinline__ void put4(void *base, int64_t at, float4 v) {
  *(typename Quad<EL>::raw *)((char *)base + at * elem_bytes(EL)) = Quad<EL>::pack(v);
}

// What four columns of a group add to a row's sums: the bias (as stored: it waits in registers),
// and for 8-bit integers the channels' scales.
template <int IN, int EL>
struct ColumnTerms {
  typename Quad<EL>::raw bias;
};
template <int EL>
struct ColumnTerms<IN_I8, EL> {
  typename Quad<EL>::raw bias;
  float scale[4];
};
template <int IN, int EL, int EPI>
__device__ __forceinline__ ColumnTerms<IN, EL> column_terms(const GluParams &p, int g, int64_t col) {
  const int64_t n = EPI == EPI_PLAIN ? p.F : 2 * p.F;
  ColumnTerms<IN, EL> c;
  if constexpr (IN == IN_I8) {
    const float *s = p.w_scale ? p.w_scale + (int64_t)g * n : p.w_scale_ptrs[g];
#pragma unroll
    for (int i = 0; i < 4; ++i) c.scale[i] = s[col + i];  // a group's scales may sit at any word
  }
  if (p.bias)
    c.bias = load_raw4<EL>(p.bias, (int64_t)g * n + col);
  else if (p.bias_ptrs)
    c.bias = load_raw4<EL>(p.bias_ptrs[g], col);
  else
    c.bias = typename Quad<EL>::raw{};
  return c;
}

// A row's scale as scale and after, whose product it is: (sum scale) channel after leaves fp32's range
// only where the whole product does (a sum is 0 or of 1 .. 2^31, so only scales past 2^96 overflow with
// it, and those leave 2^64 for the end).  The two scales' own product may leave it earlier, and 0 times
// an infinity is NaN.  The last factor is a power of two, exact, in the addition of the bias.
struct RowScale {
  float scale, after;
  __device__ __forceinline__ explicit RowScale(float s = 0.f)
      : scale(fabsf(s) > 0x1p96f ? s * 0x1p-64f : s), after(fabsf(s) > 0x1p96f ? 0x1p64f : 1.f) {}
};

template <int IN, int EL>
__device__ __forceinline__ float4 finish(typename Operand<IN>::acc_t s, const RowScale &r, const ColumnTerms<IN, EL> &c) {
  const float4 b = Quad<EL>::value(c.bias);
  if constexpr (IN == IN_I8) {
    auto one = [&](int i, float bias) { return fmaf((float)s[i] * r.scale * c.scale[i], r.after, bias); };
    return make_float4(one(0, b.x), one(1, b.y), one(2, b.z), one(3, b.w));
  } else {
    return make_float4(s[0] + b.x, s[1] + b.y, s[2] + b.z, s[3] + b.w);
  }
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
