// E4M3 / E8M0 helpers of the MXFP8 quantizers.
#pragma once

#include "gl_common.hpp"

namespace gl {

// E4M3 codes of four finite floats (already scaled into the block's range), packed
// one per byte: round to nearest even, magnitudes above 448 saturate to 448, the sign
// bit is kept (also for zero).  gfx950's pack conversion to OCP E4M3 rounds to
// nearest even and keeps the sign; the clamp first makes overflow saturate.  It gives
// the same bytes as the rule spelled out: over every bf16 value (8 significant bits,
// exponents -149 .. 9, both signs) checked exhaustively on the device, and for the
// 24-bit values of quantize_lanes at every code, every middle of two codes, the
// saturated range and one fp32 step to either side of each (tests of the RMS norm).
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  const auto sat = [](float v) { return __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f); };
  uint32_t o = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(sat(a), sat(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(sat(c), sat(d), (int)o, true);
}

// The same rule for values still in fp32, spread over the 32 / n neighbouring lanes
// that hold a block of 32: quantizes the lane's n values (n = 4 or 8) into n / 4 words
// of codes and gives the block's scale byte to every lane.  The 32 / n lanes of a block
// have to be active together.
template <int n>
__device__ __forceinline__ uint8_t quantize_lanes(const float *v, uint32_t *out) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
  for (int d = 1; d < 32 / n; d <<= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, d));
  if (amax >= 0x7f800000u) {  // Inf or NaN in the block
#pragma unroll
    for (int i = 0; i < n / 4; ++i) {
      uint32_t o = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) o |= (0x7fu | ((__float_as_uint(v[4 * i + k]) >> 24) & 0x80u)) << (8 * k);
      out[i] = o;
    }
    return 0xff;
  }
  const int ef = (int)(amax >> 23);       // biased exponent of amax (0 for zero/subnormal)
  const int byte = ef > 8 ? ef - 8 : 0;   // e + 127 with e = floor(log2 amax) - 8, e >= -127
  const float mul = __builtin_ldexpf(1.0f, 127 - byte);  // 2^-e, a normal float
#pragma unroll
  for (int i = 0; i < n / 4; ++i)
    out[i] = e4m3_pack4(v[4 * i] * mul, v[4 * i + 1] * mul, v[4 * i + 2] * mul, v[4 * i + 3] * mul);
  return (uint8_t)byte;
}

}  // namespace gl
