// Token routing of a mixture-of-experts layer: each token's top experts with their
// weights, the plan that orders the chosen (token, slot) pairs by expert for the
// grouped GEMMs, and the gradient of the weights.
//
// Selection is by logit, largest first, ties to the lowest expert; a NaN logit counts
// as -inf and a -inf logit masks its expert, which then weighs 0.  Scores: softmax over
// all experts, or the sigmoid of each logit; renormalised, a token's weights are its
// chosen scores divided by their sum (for softmax: a softmax over the chosen logits).
// A token whose experts are all masked gets weights 0.
#include "gl_vec.hpp"

namespace gl {

constexpr int kRouteThreads = 256, kRouteWaves = kRouteThreads / 64;
constexpr int kRouteMaxExperts = 1024;
constexpr int kPlanTokens = 64;  // tokens of a plan block: one bit each of a 64-bit mask

template <int EL>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
  float v;
  if constexpr (EL == EL_F32)
    v = ((const float *)p)[i];
  else
    v = h16_to_f32<EL == EL_F16>(((const uint16_t *)p)[i]);
  // NaN counts as masked; +inf as the largest finite value, so that sums stay finite
  return v != v ? -INFINITY : fminf(v, 3.402823466e38f);
}

// Unsigned order of floats without NaN, -0 equal to +0; every value maps above 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One wave a token: lane l holds experts l, l + 64, ....
template <int EL>
__global__ __launch_bounds__(kRouteThreads) void route_gates_kernel(const void *__restrict__ logits, int64_t T, int E,
                                                                    int k, int sigm, int renorm,
                                                                    int32_t *__restrict__ ids,
                                                                    float *__restrict__ weights) {
  constexpr int kPer = kRouteMaxExperts / 64;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  if (t >= T) return;
  float l[kPer];
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < E ? load_logit<EL>(logits, t * E + e) : -INFINITY;
    key[i] = e < E ? order_key(l[i]) : 0;
  }
  int my_id = 0;
  float my_l = -INFINITY;  // lane j keeps the j-th choice
  for (int j = 0; j < k; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint64_t c = ((uint64_t)key[i] << 32) | (uint32_t)~(i * 64 + lane);
      best = c > best ? c : best;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      const uint64_t o = __shfl_xor((unsigned long long)best, d);
      best = o > best ? o : best;
    }
    const int e = (int)~(uint32_t)best;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (e == i * 64 + lane) key[i] = 0;  // taken
    if (lane == j) {
      const uint32_t b = (uint32_t)(best >> 32);
      my_id = e;
      my_l = __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
    }
  }
  float w;
  if (sigm) {
    w = 1.f / (1.f + expf(-my_l));
  } else {
    const float top = __shfl(my_l, 0);
    w = top == -INFINITY ? 0.f : expf(my_l - top);
    if (!renorm) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += top == -INFINITY ? 0.f : expf(l[i] - top);
#pragma unroll
      for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
      w = sum > 0.f ? w / sum : 0.f;
    }
  }
  if (renorm) {
    float sum = lane < k ? w : 0.f;
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    w = sum > 0.f ? w / sum : 0.f;
  }
  if (lane < k) {
    ids[t * k + lane] = my_id;
    weights[t * k + lane] = w;
  }
}

// Plan.  A token names an expert at most once, so within a block of 64 tokens the
// tokens of an expert are one 64-bit mask, and a slot's rank among them is the number
// of bits below its token's.
__global__ __launch_bounds__(kRouteThreads) void route_masks_kernel(const int32_t *__restrict__ ids, int64_t T, int E,
                                                                    int k, unsigned long long *__restrict__ masks) {
  __shared__ unsigned long long m[kRouteMaxExperts];
  const int64_t t0 = (int64_t)blockIdx.x * kPlanTokens;
  const int n = (int)min64(kPlanTokens, T - t0) * k;
  for (int e = threadIdx.x; e < E; e += kRouteThreads) m[e] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < n; s += kRouteThreads) atomicOr(&m[ids[t0 * k + s]], 1ull << (s / k));
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kRouteThreads) masks[(int64_t)blockIdx.x * E + e] = m[e];
}

// One workgroup: thread e runs over the blocks of expert e, then the experts' totals
// are scanned.
__global__ __launch_bounds__(kRouteMaxExperts) void route_scan_kernel(const unsigned long long *__restrict__ masks,
                                                                      int64_t blocks, int E,
                                                                      int32_t *__restrict__ base,
                                                                      int32_t *__restrict__ start,
                                                                      int64_t *__restrict__ m_splits) {
  __shared__ int32_t tot[kRouteMaxExperts];
  const int e = threadIdx.x;
  int32_t sum = 0;
  if (e < E)
    for (int64_t b = 0; b < blocks; ++b) {
      base[b * E + e] = sum;
      sum += __popcll(masks[b * E + e]);
    }
  tot[e] = e < E ? sum : 0;
  __syncthreads();
  for (int d = 1; d < kRouteMaxExperts; d <<= 1) {
    const int32_t v = e >= d ? tot[e - d] : 0;
    __syncthreads();
    tot[e] += v;
    __syncthreads();
  }
  if (e < E) {
    start[e] = tot[e] - sum;
    m_splits[e] = sum;
  }
}

__global__ __launch_bounds__(kRouteThreads) void route_rows_kernel(const int32_t *__restrict__ ids, int64_t T, int E,
                                                                   int k, const unsigned long long *__restrict__ masks,
                                                                   const int32_t *__restrict__ base,
                                                                   const int32_t *__restrict__ start,
                                                                   int32_t *__restrict__ row_index,
                                                                   int32_t *__restrict__ slot_index) {
  const int64_t t0 = (int64_t)blockIdx.x * kPlanTokens;
  const int n = (int)min64(kPlanTokens, T - t0) * k;
  for (int s = threadIdx.x; s < n; s += kRouteThreads) {
    const int e = ids[t0 * k + s];
    const int64_t at = (int64_t)blockIdx.x * E + e;
    const int row = start[e] + base[at] + __popcll(masks[at] & ((1ull << (s / k)) - 1));
    row_index[t0 * k + s] = row;
    slot_index[row] = (int32_t)(t0 * k + s);
  }
}

// Gradient of the weights, one wave a token.  With s the scores before any division
// and w = s / sum(s) where renormalised:
//   softmax             dl_e = p_e (dw_e - sum_j dw_j p_j)        (dw_e 0 if not chosen)
//   softmax, renorm.    dl_j = w_j (dw_j - sum_i dw_i w_i)        (chosen only)
//   sigmoid             dl_j = dw_j s_j (1 - s_j)
//   sigmoid, renorm.    dl_j = (1 - s_j) w_j (dw_j - sum_i dw_i w_i)
template <int EL>
__global__ __launch_bounds__(kRouteThreads) void route_bwd_kernel(const void *__restrict__ logits, int64_t T, int E,
                                                                  int k, int sigm, int renorm,
                                                                  const int32_t *__restrict__ ids,
                                                                  const float *__restrict__ dweights,
                                                                  void *__restrict__ dlogits) {
  constexpr int kPer = kRouteMaxExperts / 64;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  if (t >= T) return;
  const auto sum = [](float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
  };
  float l[kPer], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < E ? load_logit<EL>(logits, t * E + e) : -INFINITY;
    top = fmaxf(top, l[i]);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  // lane j holds slot j; an id outside the experts takes no part
  int id = -1;
  float dw = 0.f, s = 0.f, slope = 1.f;
  if (lane < k) {
    id = ids[t * k + lane];
    if (id < 0 || id >= E) id = -1;
    dw = dweights[t * k + lane];
  }
  if (id >= 0) {
    const float v = load_logit<EL>(logits, t * E + id);
    if (sigm) {
      s = 1.f / (1.f + expf(-v));
      slope = 1.f - s;
    } else {
      s = top == -INFINITY ? 0.f : expf(v - top);
    }
  }
  float total = 1.f;
  if (renorm)
    total = sum(s);
  else if (!sigm) {
    total = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) total += top == -INFINITY ? 0.f : expf(l[i] - top);
    total = sum(total);
  }
  const float w = total > 0.f ? s / total : 0.f;
  const float mean = !sigm || renorm ? sum(id >= 0 ? dw * w : 0.f) : 0.f;
  const float mine = id >= 0 ? slope * w * (dw - mean) : 0.f;
  // every expert's value: chosen from its slot, others 0 or their share of the softmax
  const bool dense = !sigm && !renorm;
  float o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    o[i] = dense && total > 0.f ? -mean * (expf(l[i] - top) / total) : 0.f;
  for (int j = 0; j < k; ++j) {
    const int e = __shfl(id, j);
    const float v = __shfl(mine, j);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (e == i * 64 + lane) o[i] = v;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * 64 + lane;
    if (e >= E) break;
    if constexpr (EL == EL_F32)
      ((float *)dlogits)[t * E + e] = o[i];
    else
      ((uint16_t *)dlogits)[t * E + e] = f32_to_h16<EL == EL_F16>(o[i]);
  }
}

struct RoutePlan {
  unsigned long long *masks;  // [blocks][E]
  int32_t *base;              // [blocks][E]
  int32_t *start;             // [E]
};

size_t route_plan_bytes(int64_t T, int E) {
  const int64_t blocks = (T + kPlanTokens - 1) / kPlanTokens;
  return (size_t)(blocks * E * 12 + E * 4 + 15) & ~(size_t)15;
}

hipError_t launch_route_fwd(int el, int64_t T, int E, int k, int sigm, int renorm, const void *logits, int32_t *ids,
                            float *weights, int64_t *m_splits, int32_t *row_index, int32_t *slot_index, void *ws,
                            hipStream_t s) {
  const int64_t blocks = (T + kPlanTokens - 1) / kPlanTokens;
  const dim3 grid((unsigned)((T + kRouteWaves - 1) / kRouteWaves)), block(kRouteThreads);
  if (T > 0) {
    if (el == EL_F32)
      hipLaunchKernelGGL(route_gates_kernel<EL_F32>, grid, block, 0, s, logits, T, E, k, sigm, renorm, ids, weights);
    else if (el == EL_F16)
      hipLaunchKernelGGL(route_gates_kernel<EL_F16>, grid, block, 0, s, logits, T, E, k, sigm, renorm, ids, weights);
    else
      hipLaunchKernelGGL(route_gates_kernel<EL_BF16>, grid, block, 0, s, logits, T, E, k, sigm, renorm, ids, weights);
  }
  if (m_splits) {
    RoutePlan r;
    r.masks = (unsigned long long *)ws;
    r.base = (int32_t *)(r.masks + blocks * E);
    r.start = r.base + blocks * E;
    if (T > 0)
      hipLaunchKernelGGL(route_masks_kernel, dim3((unsigned)blocks), block, 0, s, ids, T, E, k, r.masks);
    hipLaunchKernelGGL(route_scan_kernel, dim3(1), dim3(kRouteMaxExperts), 0, s, r.masks, blocks, E, r.base, r.start,
                       m_splits);
    if (T > 0)
      hipLaunchKernelGGL(route_rows_kernel, dim3((unsigned)blocks), block, 0, s, ids, T, E, k, r.masks, r.base,
                         r.start, row_index, slot_index);
  }
  return hipGetLastError();
}

hipError_t launch_route_bwd(int el, int64_t T, int E, int k, int sigm, int renorm, const void *logits,
                            const int32_t *ids, const float *dweights, void *dlogits, hipStream_t s) {
  const dim3 grid((unsigned)((T + kRouteWaves - 1) / kRouteWaves)), block(kRouteThreads);
  if (el == EL_F32)
    hipLaunchKernelGGL(route_bwd_kernel<EL_F32>, grid, block, 0, s, logits, T, E, k, sigm, renorm, ids, dweights,
                       dlogits);
  else if (el == EL_F16)
    hipLaunchKernelGGL(route_bwd_kernel<EL_F16>, grid, block, 0, s, logits, T, E, k, sigm, renorm, ids, dweights,
                       dlogits);
  else
    hipLaunchKernelGGL(route_bwd_kernel<EL_BF16>, grid, block, 0, s, logits, T, E, k, sigm, renorm, ids, dweights,
                       dlogits);
  return hipGetLastError();
}

}  // namespace gl
