// 16-byte vectors of a tensor's elements as fp32 values, shared by the kernels that
// stream rows (SwiGLU, the RMS norm, the expert layer for a few tokens).
#pragma once

#include "gl_common.hpp"

namespace gl {

// element type of a streamed tensor
enum { EL_BF16 = 0, EL_F32 = 1, EL_F16 = 2 };

template <int EL>
struct Vec;  // 16 bytes of elements <-> fp32 values

template <>
struct Vec<EL_F32> {
  static constexpr int n = 4;
  __device__ static void load(const void *p, float *v) {
    const float4 q = *(const float4 *)p;
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  }
  __device__ static void store(void *p, const float *v) { *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]); }
};

template <int EL>
struct Vec16 {
  static constexpr int n = 8;
  static constexpr bool F16 = EL == EL_F16;
  __device__ static void load(const void *p, float *v) {
    const uint4 q = *(const uint4 *)p;
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = h16_to_f32<F16>((uint16_t)(w[i] & 0xffffu));
      v[2 * i + 1] = h16_to_f32<F16>((uint16_t)(w[i] >> 16));
    }
  }
  __device__ static void store(void *p, const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = pack_h16x2<F16>(v[2 * i], v[2 * i + 1]);
    *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<EL_BF16> : Vec16<EL_BF16> {};
template <>
struct Vec<EL_F16> : Vec16<EL_F16> {};

// A launch may have fewer than 2^32 threads: grids that grow with the rows go out in slices of
// at most this many.
constexpr int64_t kSliceThreads = (int64_t)1 << 31;

constexpr int elem_bytes(int el) { return el == EL_F32 ? 4 : 2; }

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + __expf(-v)); }

}  // namespace gl
