// Token routing of a mixture-of-experts layer: each token's top experts with their
// weights, the plan that orders the chosen (token, slot) pairs by expert for the
// grouped GEMMs, and the gradient of the weights.
//
// Selection is by logit, largest first, ties to the lowest expert; a NaN logit counts
// as -inf and a -inf logit masks its expert, which then weighs 0.  Scores: softmax over
// all experts, or the sigmoid of each logit; renormalised, a token's weights are its
// chosen scores divided by their sum (for softmax: a softmax over the chosen logits).
// A token whose experts are all masked gets weights 0.
//
// 32768 tokens over 256 experts, bf16, top 8: gates 14.3 us, scan 4.7, rows 5.2 (21 MB in
// all); 32 tokens over 64 experts with their plan, one launch, 4.1 us; the gradient of
// 16384 x 64 fp32 6.3 us (5.0 out of the last-level cache).
#include <type_traits>

#include "gl_vec.hpp"

namespace gl {

constexpr int kRouteMaxExperts = 1024, kRouteMaxTopK = 32;
constexpr int kChunk = 64;  // tokens of a workgroup: one bit each of a 64-bit mask
constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;

__device__ __forceinline__ float as_logit(float v) {
  // NaN counts as masked; +inf as the largest finite value, so that sums stay finite
  return v != v ? -INFINITY : fminf(v, 3.402823466e38f);
}

template <int EL>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
  if constexpr (EL == EL_F32) return as_logit(((const float *)p)[i]);
  else return as_logit(h16_to_f32<EL == EL_F16>(((const uint16_t *)p)[i]));
}

// sigmoid(v) e^-base, base at most 0 (and 0 where any v of the row is above): without overflow
// of e^-v, and with the base of score_base no sum of a row's scores underflows.
__device__ __forceinline__ float sigmoid_score(float v, float base) {
  return (v > 0.f ? 1.f : expf(v - base)) / (1.f + expf(-fabsf(v)));
}
// The base for scores that are divided by their sum, from the largest logit among them.  Below
// -745, where 64 bits hold its sigmoid as 0, a logit is a mask (a type's lowest value, say):
// scores stay 0.
__device__ __forceinline__ float score_base(float largest) { return largest > -745.f ? fminf(largest, 0.f) : 0.f; }

// Unsigned order of floats without NaN, -0 equal to +0; every value maps above 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A token's row is held by LPR lanes, PER consecutive experts each: 16 lanes (four tokens a
// wave, reductions by four rotations within 16 lanes) up to 256 experts, else the wave.
template <int LPR_, int PER_>
struct RowLanes {
  static constexpr int LPR = LPR_, PER = PER_, rows = 64 / LPR_;  // rows of a wave
};

template <int ror>
__device__ __forceinline__ uint32_t rotate16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + ror, 0xf, 0xf, true);
}

// f over the LPR lanes of the row, in every lane of it
template <int LPR, class F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, F f) {
  v = f(v, rotate16<8>(v));
  v = f(v, rotate16<4>(v));
  v = f(v, rotate16<2>(v));
  v = f(v, rotate16<1>(v));
  if constexpr (LPR == 64) {
    v = f(v, (uint32_t)__shfl_xor((int)v, 16));
    v = f(v, (uint32_t)__shfl_xor((int)v, 32));
  }
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  return __uint_as_float(row_reduce<LPR>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

template <int LPR>
__device__ __forceinline__ float row_max_float(float v) {
  return __uint_as_float(row_reduce<LPR>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  return row_reduce<LPR>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int LPR>
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  return row_reduce<LPR>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

// The lane's experts as keys in the order of choice, and a round of it: the row's best
// expert still there.  No key but a missing expert's is 0.
template <int EL, int LPR, int PER>
struct Choices {
  uint32_t key[PER], last = 0;
  int e0;
  __device__ Choices(const float *l, int e0_, int E) : e0(e0_) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      uint32_t k;
      if constexpr (EL == EL_F32) {
        k = order_key(l[i]);
      } else {
        // the value's own 16 bits in order, and below them a larger number for a lower
        // expert: all keys of a row differ
        const uint32_t b = f32_to_h16<EL == EL_F16>(l[i] + 0.f);
        k = ((b & 0x8000u ? ~b & 0xffffu : b | 0x8000u) << 16) | (uint32_t)(0xffff - e0 - i);
      }
      key[i] = e0 + i < E ? k : 0;
    }
  }
  // every lane of the row gets the choice's key and expert
  __device__ void next(uint32_t &m, int &e) {
    uint32_t best = 0;
    if constexpr (EL == EL_F32) {
#pragma unroll
      for (int i = 0; i < PER; ++i) best = key[i] > best ? key[i] : best;
      m = row_max<LPR>(best);
      uint32_t at = 0xffffffffu;  // the lowest expert of that key
#pragma unroll
      for (int i = PER - 1; i >= 0; --i) at = key[i] == m ? e0 + i : at;
      e = (int)row_min<LPR>(at);
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = e == e0 + i ? 0 : key[i];
    } else {
      // the keys differ, so the next is the largest below the last: modulo 2^32 the keys
      // below it are the ones of the largest differences to it (at first, to 0, all are)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint32_t d = key[i] - last;
        best = d > best ? d : best;
      }
      m = last + row_max<LPR>(best);
      last = m;
      e = 0xffff - (int)(m & 0xffff);
    }
  }
  // the logit of a choice's key
  __device__ static float logit(uint32_t m) {
    if constexpr (EL == EL_F32) return __uint_as_float(m & 0x80000000u ? m & 0x7fffffffu : ~m);
    const uint32_t b = m >> 16;
    return as_logit(h16_to_f32<EL == EL_F16>((uint16_t)(b & 0x8000u ? b & 0x7fffu : ~b)));
  }
};

// The lane's PER logits of row t from expert e0 on, -inf past the experts.  whole: rows
// start on a multiple of the loads' 16 (or, 4 values of 16 bits, 8) bytes.
template <int EL, int PER>
__device__ __forceinline__ void load_row(const void *logits, int64_t t, int E, int e0, bool whole, float *l) {
  constexpr int V = EL == EL_F32 ? 4 : PER < 8 ? 4 : 8;  // values of a load
  if (whole) {
#pragma unroll
    for (int i = 0; i < PER; i += V) {
      if (e0 + i >= E) {
#pragma unroll
        for (int j = 0; j < V; ++j) l[i + j] = -INFINITY;
        continue;
      }
      if constexpr (EL == EL_F32) {
        const float4 q = *(const float4 *)((const float *)logits + t * E + e0 + i);
        l[i] = as_logit(q.x); l[i + 1] = as_logit(q.y); l[i + 2] = as_logit(q.z); l[i + 3] = as_logit(q.w);
      } else {
        uint32_t w[V / 2];
        const uint16_t *at = (const uint16_t *)logits + t * E + e0 + i;
        if constexpr (V == 8) __builtin_memcpy(w, __builtin_assume_aligned(at, 16), 16);
        else __builtin_memcpy(w, __builtin_assume_aligned(at, 8), 8);
#pragma unroll
        for (int j = 0; j < V; ++j)
          l[i + j] = as_logit(h16_to_f32<EL == EL_F16>((uint16_t)(w[j / 2] >> (16 * (j & 1)))));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = e0 + i < E ? load_logit<EL>(logits, t * E + e0 + i) : -INFINITY;
  }
}

// Inclusive sums over the wave's lanes, and over a workgroup of kRouteThreads.
__device__ __forceinline__ int wave_scan(int v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if ((int)(threadIdx.x & 63) >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ int block_scan(int v) {
  __shared__ int waves[kRouteWaves];
  v = wave_scan(v);
  if ((threadIdx.x & 63) == 63) waves[threadIdx.x >> 6] = v;
  __syncthreads();
  for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) v += waves[w];
  return v;
}

struct RouteForward {
  const void *logits;
  int32_t *ids;
  float *weights;
  unsigned long long *masks;  // [chunks][E] tokens of the chunk that chose the expert, or null
  int64_t *m_splits;
  int32_t *row_index, *slot_index;
  int64_t T, chunk0;  // chunk0: of the launch's first workgroup
  int E, k, sigm, renorm, whole;
};

// Gates of a chunk of 64 tokens, and the chunk's part of the plan.  A token names an
// expert at most once, so the chunk's tokens of an expert are one 64-bit mask, and a
// slot's rank among them is the number of bits below its token's.  A call of one chunk
// makes its whole plan here.
//
// Bound by instructions and, for few tokens, latency: k rounds over the keys that the
// row's lanes hold.  (Sorting each lane's keys first, so that a round looks at one, took
// four times as long with keys of 64 bits, value and expert; with the 32-bit keys that
// 16-bit logits have now it has not been tried.)
template <int EL, class R>
__global__ __launch_bounds__(kRouteThreads) void route_gates_kernel(const RouteForward p) {
  constexpr int LPR = R::LPR, PER = R::PER, H = LPR == 64 ? 1 : 2;
  __shared__ unsigned long long mask[kRouteMaxExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane / LPR, pos = lane % LPR;
  const int64_t chunk = p.chunk0 + blockIdx.x, t0 = chunk * kChunk;
  const int e0 = pos * PER, k = p.k;
  constexpr int kRounds = kChunk / (kRouteWaves * R::rows);
  int id[kRounds][H];  // the row's lane j keeps choices j and, of 16 lanes, 16 + j; -1: none
  if (p.m_splits)
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) mask[e] = 0;
#pragma unroll
  for (int round = 0; round < kRounds; ++round) {
    const int r = (round * kRouteWaves + wave) * R::rows + sub;
    const int64_t t = t0 + r;
#pragma unroll
    for (int h = 0; h < H; ++h) id[round][h] = -1;
    if (t >= p.T) continue;
    float l[PER];
    load_row<EL, PER>(p.logits, t, p.E, e0, p.whole, l);
    Choices<EL, LPR, PER> choices(l, e0, p.E);
    uint32_t key[H] = {};
    for (int j = 0; j < k; ++j) {
      uint32_t m;
      int e;
      choices.next(m, e);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const bool mine = j == h * LPR + pos;
        key[h] = mine ? m : key[h];
        id[round][h] = mine ? e : id[round][h];
      }
    }
    // scores of the choices, and of all where they are divided by their sum
    const float top = choices.logit((uint32_t)__shfl((int)key[0], sub * LPR));
    const float base = p.renorm ? score_base(top) : 0.f;
    float w[H], sum = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const float v = choices.logit(key[h]);
      w[h] = h * LPR + pos >= k ? 0.f : p.sigm ? sigmoid_score(v, base) : top == -INFINITY ? 0.f : expf(v - top);
      sum += w[h];
    }
    if (p.renorm) {
      sum = row_sum<LPR>(sum);
    } else if (p.sigm) {
      sum = 1.f;
    } else {
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += top == -INFINITY ? 0.f : expf(l[i] - top);
      sum = row_sum<LPR>(sum);
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int j = h * LPR + pos;
      if (j < k) {
        p.ids[t * k + j] = id[round][h];
        p.weights[t * k + j] = sum > 0.f ? w[h] / sum : 0.f;
      }
    }
  }
  if (!p.m_splits) return;
  const auto each_slot = [&](auto f) {  // f(token of the chunk, slot, expert)
#pragma unroll
    for (int round = 0; round < kRounds; ++round)
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (id[round][h] >= 0) f((round * kRouteWaves + wave) * R::rows + sub, h * LPR + pos, id[round][h]);
  };
  __syncthreads();
  each_slot([&](int r, int, int e) { atomicOr(&mask[e], 1ull << r); });
  __syncthreads();
  if (p.T > kChunk) {
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) p.masks[chunk * p.E + e] = mask[e];
    return;
  }
  // the only chunk: an expert's rows start at the sum of the counts before it
  __shared__ int start[kRouteMaxExperts];
  const int e = threadIdx.x, n = e < p.E ? __popcll(mask[e]) : 0;
  start[e] = block_scan(n) - n;
  if (e < p.E) p.m_splits[e] = n;
  __syncthreads();
  each_slot([&](int r, int j, int e) {
    const int row = start[e] + __popcll(mask[e] & ((1ull << r) - 1)), s = r * k + j;
    p.row_index[s] = row;
    p.slot_index[row] = s;
  });
}

// Where a chunk's slots of an expert start among the expert's.  A workgroup takes 16
// experts, neighbours in every chunk's masks, and splits the chunks into 64 runs: thread
// (run, expert) adds up its run, the runs' sums are scanned, and it goes over its run again.
__global__ __launch_bounds__(kRouteThreads) void route_scan_kernel(const unsigned long long *__restrict__ masks,
                                                                   int64_t chunks, int E, int32_t *__restrict__ base,
                                                                   int64_t *__restrict__ m_splits) {
  static_assert(kRouteWaves == 16, "a wave scans one of the workgroup's experts");
  __shared__ int sums[64][17];
  const int col = threadIdx.x & 15, run = threadIdx.x >> 4, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 16 + col;
  const int64_t per = (chunks + 63) / 64, c0 = run * per, c1 = e < E ? min64(c0 + per, chunks) : 0;
  int n = 0;
#pragma unroll 8
  for (int64_t c = c0; c < c1; ++c) n += __popcll(masks[c * E + e]);
  sums[run][col] = n;
  __syncthreads();
  const int v = sums[lane][wave], upto = wave_scan(v);
  sums[lane][wave] = upto - v;
  if (lane == 63 && blockIdx.x * 16 + wave < E) m_splits[blockIdx.x * 16 + wave] = upto;
  __syncthreads();
  n = sums[run][col];
#pragma unroll 8
  for (int64_t c = c0; c < c1; ++c) {
    base[c * E + e] = n;
    n += __popcll(masks[c * E + e]);
  }
}

// The rows of a chunk's slots: the experts' starts (a scan of the totals, made by every
// workgroup), the chunk's within the expert, and the rank within the chunk.
__global__ __launch_bounds__(kRouteThreads) void route_rows_kernel(const int32_t *__restrict__ ids, int64_t T,
                                                                   int64_t chunk0, int E, int k,
                                                                   const unsigned long long *__restrict__ masks,
                                                                   const int32_t *__restrict__ base,
                                                                   const int64_t *__restrict__ m_splits,
                                                                   int32_t *__restrict__ row_index,
                                                                   int32_t *__restrict__ slot_index) {
  __shared__ int start[kRouteMaxExperts];
  __shared__ unsigned long long mask[kRouteMaxExperts];
  const int64_t chunk = chunk0 + blockIdx.x, t0 = chunk * kChunk;
  const int n = (int)min64(kChunk, T - t0) * k;
  constexpr int kSlots = kChunk * kRouteMaxTopK / kRouteThreads;  // slots of a thread
  int id[kSlots];  // loaded with the tables, so that the scan does not wait twice
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int s = i * kRouteThreads + threadIdx.x;
    id[i] = s < n ? ids[t0 * k + s] : -1;
  }
  const int e = threadIdx.x;
  int total = 0, here = 0;
  if (e < E) {
    total = (int)m_splits[e];
    here = base[chunk * E + e];
    mask[e] = masks[chunk * E + e];
  }
  start[e] = block_scan(total) - total + here;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int s = i * kRouteThreads + threadIdx.x;
    if (id[i] < 0) continue;
    const int row = start[id[i]] + __popcll(mask[id[i]] & ((1ull << (s / k)) - 1));
    row_index[t0 * k + s] = row;
    slot_index[row] = (int32_t)(t0 * k + s);
  }
}

struct RouteBackward {
  const void *logits;
  const int32_t *ids;
  const float *dweights;
  void *dlogits;
  int64_t T;
  int E, k, sigm, renorm, whole;
};

// Gradient of the weights.  With s the scores before any division and w = s / sum(s) where
// renormalised:
//   softmax             dl_e = p_e (dw_e - sum_j dw_j p_j)        (dw_e 0 if not chosen)
//   softmax, renorm.    dl_j = w_j (dw_j - sum_i dw_i w_i)        (chosen only)
//   sigmoid             dl_j = dw_j s_j (1 - s_j)
//   sigmoid, renorm.    dl_j = (1 - s_j) w_j (dw_j - sum_i dw_i w_i)
template <int EL, class R>
__global__ __launch_bounds__(256) void route_bwd_kernel(const RouteBackward p) {
  constexpr int LPR = R::LPR, PER = R::PER, H = LPR == 64 ? 1 : 2;
  const int lane = threadIdx.x & 63, sub = lane / LPR, pos = lane % LPR, e0 = pos * PER, k = p.k;
  const int64_t t = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * R::rows + sub;
  const bool in = t < p.T;  // (every lane stays for the row's reductions)
  float l[PER], top = -INFINITY;
  if (in) {
    load_row<EL, PER>(p.logits, t, p.E, e0, p.whole, l);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
  top = row_max_float<LPR>(top);
  // the row's lane j holds slots j and LPR + j; an id outside the experts takes no part
  int id[H];
  float dw[H], s[H], slope[H], v[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int j = h * LPR + pos;
    id[h] = -1;
    dw[h] = 0.f;
    v[h] = -INFINITY;
    if (in && j < k) {
      const int e = p.ids[t * k + j];
      if (e >= 0 && e < p.E) {
        id[h] = e;
        const float d = p.dweights[t * k + j];
        v[h] = load_logit<EL>(p.logits, t * p.E + e);
        dw[h] = v[h] > -INFINITY ? d : 0.f;  // a masked slot's may be anything, NaN too
      }
    }
  }
  float base = 0.f;
  if (p.sigm && p.renorm) {
    base = -INFINITY;
#pragma unroll
    for (int h = 0; h < H; ++h) base = fmaxf(base, v[h]);
    base = score_base(row_max_float<LPR>(base));
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
    s[h] = p.sigm ? sigmoid_score(v[h], base) : top == -INFINITY ? 0.f : expf(v[h] - top);
    slope[h] = p.sigm ? 1.f / (1.f + expf(v[h])) : 1.f;  // 1 - s would cancel: nothing is left of it from 17 on
  }
  const bool dense = !p.sigm && !p.renorm;  // every expert has a share
  float x[PER], total = 1.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = 0.f;
  if (p.renorm) {
    total = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h) total += s[h];
    total = row_sum<LPR>(total);
  } else if (dense) {
    total = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      x[i] = top == -INFINITY ? 0.f : expf(l[i] - top);
      total += x[i];
    }
    total = row_sum<LPR>(total);
  }
  float mean = 0.f, mine[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    s[h] = total > 0.f ? s[h] / total : 0.f;
    mean += dw[h] * s[h];
  }
  mean = p.sigm && !p.renorm ? 0.f : row_sum<LPR>(mean);
#pragma unroll
  for (int h = 0; h < H; ++h) mine[h] = id[h] >= 0 ? slope[h] * s[h] * (dw[h] - mean) : 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = dense && total > 0.f ? -mean * (x[i] / total) : 0.f;
  for (int j = 0; j < k; ++j) {
    const int src = sub * LPR + j % LPR;
    const int e = __shfl(H == 2 && j >= LPR ? id[H - 1] : id[0], src);
    const float v = __shfl(H == 2 && j >= LPR ? mine[H - 1] : mine[0], src);
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = e == e0 + i ? v : x[i];
  }
  if (!in) return;
  const int64_t at = t * p.E + e0;
  if (p.whole) {
    constexpr int V = EL == EL_F32 ? 4 : PER < 8 ? 4 : 8;
#pragma unroll
    for (int i = 0; i < PER; i += V) {
      if (e0 + i >= p.E) continue;
      if constexpr (EL == EL_F32) {
        *(float4 *)((float *)p.dlogits + at + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      } else {
        uint32_t w[V / 2];
#pragma unroll
        for (int j = 0; j < V; j += 2) w[j / 2] = pack_h16x2<EL == EL_F16>(x[i + j], x[i + j + 1]);
        uint16_t *o = (uint16_t *)p.dlogits + at + i;
        if constexpr (V == 8) __builtin_memcpy(__builtin_assume_aligned(o, 16), w, 16);
        else __builtin_memcpy(__builtin_assume_aligned(o, 8), w, 8);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (e0 + i >= p.E) continue;
      if constexpr (EL == EL_F32) ((float *)p.dlogits)[at + i] = x[i];
      else ((uint16_t *)p.dlogits)[at + i] = f32_to_h16<EL == EL_F16>(x[i]);
    }
  }
}

size_t route_plan_bytes(int64_t T, int E) {
  const int64_t chunks = (T + kChunk - 1) / kChunk;
  return (size_t)(chunks * E * 12 + 31) & ~(size_t)15;
}

// f(element type, lanes and experts a lane of a row)
template <class F>
static void each_route(int el, int E, F f) {
  const auto rows = [&](auto e) {
    if (E <= 64) f(e, RowLanes<16, 4>());
    else if (E <= 128) f(e, RowLanes<16, 8>());
    else if (E <= 256) f(e, RowLanes<16, 16>());
    else f(e, RowLanes<64, 16>());
  };
  if (el == EL_F32) rows(std::integral_constant<int, EL_F32>());
  else if (el == EL_F16) rows(std::integral_constant<int, EL_F16>());
  else rows(std::integral_constant<int, EL_BF16>());
}

// Whether load_row's loads are aligned in every row.
static int whole_rows(int el, int E) { return E % (el == EL_F32 || E <= 64 ? 4 : 8) == 0; }

hipError_t launch_route_fwd(int el, int64_t T, int E, int k, int sigm, int renorm, const void *logits, int32_t *ids,
                            float *weights, int64_t *m_splits, int32_t *row_index, int32_t *slot_index, void *ws,
                            hipStream_t s) {
  const int64_t chunks = (T + kChunk - 1) / kChunk;
  RouteForward p{logits, ids, weights, (unsigned long long *)ws, m_splits, row_index, slot_index,
                 T, 0, E, k, sigm, renorm, whole_rows(el, E)};
  const dim3 block(kRouteThreads);
  // f(first chunk, workgroups) of every slice of the chunks (no tokens: one workgroup writes
  // the counts)
  const auto slices = [&](auto f) {
    constexpr int64_t step = kSliceThreads / kRouteThreads;
    for (int64_t c = 0; c == 0 || c < chunks; c += step) f(c, dim3((unsigned)(chunks ? min64(chunks - c, step) : 1)));
  };
  each_route(el, E, [&](auto e, auto r) {
    slices([&](int64_t c, dim3 grid) {
      p.chunk0 = c;
      hipLaunchKernelGGL((route_gates_kernel<e(), decltype(r)>), grid, block, 0, s, p);
    });
  });
  if (m_splits && chunks > 1) {
    int32_t *base = (int32_t *)(p.masks + chunks * E);
    hipLaunchKernelGGL(route_scan_kernel, dim3((unsigned)((E + 15) / 16)), block, 0, s, p.masks,
                       chunks, E, base, m_splits);
    slices([&](int64_t c, dim3 grid) {
      hipLaunchKernelGGL(route_rows_kernel, grid, block, 0, s, ids, T, c, E, k, p.masks, base, m_splits, row_index,
                         slot_index);
    });
  }
  return hipGetLastError();
}

hipError_t launch_route_bwd(int el, int64_t T, int E, int k, int sigm, int renorm, const void *logits,
                            const int32_t *ids, const float *dweights, void *dlogits, hipStream_t s) {
  each_route(el, E, [&](auto e, auto r) {
    constexpr int64_t rows = 4 * decltype(r)::rows, step = kSliceThreads / 256 * rows;
    const int64_t row = (int64_t)E * elem_bytes(e());
    for (int64_t t = 0; t < T; t += step) {
      const int64_t n = min64(T - t, step);
      const RouteBackward p{(const char *)logits + t * row, ids + t * k, dweights + t * k, (char *)dlogits + t * row,
                            n, E, k, sigm, renorm, whole_rows(el, E)};
      hipLaunchKernelGGL((route_bwd_kernel<e(), decltype(r)>), dim3((unsigned)((n + rows - 1) / rows)), dim3(256), 0,
                         s, p);
    }
  });
  return hipGetLastError();
}

}  // namespace gl
