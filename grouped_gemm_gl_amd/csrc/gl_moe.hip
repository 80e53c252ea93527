// The expert layer for a few tokens: for token t with experts e_j = ids[t, j] and
// weights w_j
//   y_t = residual_t + sum_j w_j (W2_e SwiGLU(W1_e x_t + b1_e) + b2_e)
// in two kernels, without sorting or gathering rows.  A slot whose id is no expert of
// this call, or whose weight is 0, takes no part.
//
// Both are bound by reading the used experts' weights once from HBM, so both stream
// weight rows straight from global memory into the A operand of 16-row MFMA steps (no
// LDS in between: no workgroup shares a weight with another) and take the few tokens as
// the B operand's columns from cache.
//
//   up    workgroup (expert, 16 columns of a): the expert's tokens, compacted, are the
//         columns; its waves split the contraction over K and add up through LDS.  Leaves
//         a = w SwiGLU(W1 x + b1), w the token's weight for the expert, in the workspace.
//   down  workgroup (16 columns of y): runs over all (expert, piece of F) items of the
//         call with the tokens themselves as columns, a column without the expert being
//         zeros, so the sum over a token's experts is the MFMA's own accumulation: one
//         accumulator a token, no atomics, a fixed order.
//
// For 16-bit weights a is kept as two values of the weights' type, the rounded value and
// the rest, each multiplied in its own MFMA step: the products see 16 significant bits
// of a (22 for fp16) where one value would add its own rounding, of the output's size,
// to the result.  The extra step is free beside the weight read.
#include <type_traits>

#include "gl_vec.hpp"

namespace gl {

constexpr int kMoeMaxTokens = 64;
constexpr int kUpThreads = 256, kUpWaves = kUpThreads / 64;
constexpr int kDownThreads = 512, kDownWaves = kDownThreads / 64;
constexpr int kMoeRows = 16;  // weight rows of a workgroup (per half of W1)
enum { EL_MX = 3 };           // weights: E4M3 codes with an E8M0 scale per 32 of a row

struct MoeWeight {
  const char *w;
  const char *const *w_ptrs;
  const uint8_t *scale;
  const uint8_t *const *scale_ptrs;
  const char *bias;
  const char *const *bias_ptrs;
  int64_t rows, cols;  // of one expert's matrix
};

// An expert with its tokens, written by the up kernel: at most one per slot, and one per
// expert.
struct MoeEntry {
  int32_t expert;  // -1: none
  int32_t pad;
  uint64_t tokens;  // bit t: token t has a slot of it
};

struct MoeParams {
  const char *x;
  const int32_t *ids;
  const float *gates;
  MoeWeight w1, w2;
  const char *residual;
  char *y;
  MoeEntry *entries;  // [min(T k, E)]
  int16_t *slot_of;   // [entries][64] slot whose row of a holds a token's values
  char *a;            // [T k][F] fp32, or two planes [T k][F] of the 16-bit type
  int T, k, E, n_entries;
  int64_t K, F, N;
};

// Bytes of the workspace before `a`.
__host__ __device__ inline size_t moe_table_bytes(int n) { return (size_t)n * (sizeof(MoeEntry) + 64 * 2); }

// A lane's buffer offset that lies past every resource: the load gives zeros.
constexpr uint32_t kNowhere = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t moe_rsrc(const void *base) {
  const uint64_t v = (uint64_t)(uintptr_t)base;  // the same in every lane; made visibly so
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void *)(uintptr_t)(((uint64_t)hi << 32) | lo), (short)0, 0x7fffffff,
                                           0x00020000);
}

__device__ __forceinline__ i32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

__device__ __forceinline__ float e8m0(uint32_t s) {
  return __uint_as_float(s == 0xff ? 0x7fc00000u : s ? s << 23 : 0x00400000u);
}

// A unit is 128 bytes of each of the 16 weight rows: lane l holds bytes 16 (l / 16) and
// 64 + 16 (l / 16) of row l % 16, two loads that together take whole lines.  Its k values
// are taken in the order that this gives, the same for both operands, in `steps` pieces:
// piece i contracts the 16 bytes that b_byte(i) names of each token's row.
template <int WEL>
struct Unit {  // bf16, fp16 and fp32 weights
  static constexpr int kElems = 128 / elem_bytes(WEL);
  static constexpr int steps = 2;
  static constexpr int b_bytes = 128;  // of a token's row
  i32x4_t r[2];
  __device__ static uint32_t b_byte(int i, int q) { return i * 64 + q * 16; }
  // row: byte offset of the lane's row, at: byte within it, end: bytes of a row
  __device__ void load(__amdgpu_buffer_rsrc_t w, __amdgpu_buffer_rsrc_t, uint32_t row, uint32_t at, uint32_t end,
                       uint32_t, int q) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t b = at + i * 64 + q * 16;
      r[i] = load16(w, b < end ? row + b : kNowhere);
    }
  }
  __device__ i32x4_t operand(int i) const { return r[i]; }
};

template <>
struct Unit<EL_MX> {
  static constexpr int kElems = 128;
  static constexpr int steps = 4;
  static constexpr int b_bytes = 256;
  i32x4_t r[2];
  uint8_t s[2];
  __device__ static uint32_t b_byte(int i, int q) { return (i >> 1) * 128 + q * 32 + (i & 1) * 16; }
  __device__ void load(__amdgpu_buffer_rsrc_t w, __amdgpu_buffer_rsrc_t sc, uint32_t row, uint32_t at, uint32_t end,
                       uint32_t srow, int q) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t b = at + i * 64 + q * 16;
      r[i] = load16(w, b < end ? row + b : kNowhere);
      s[i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(sc, (int)(b < end ? srow + b / 32 : kNowhere), 0, 0);
    }
  }
  // 8 codes as bf16: their values are exact there
  __device__ i32x4_t operand(int i) const {
    const float f = e8m0(s[i >> 1]);
    i32x4_t o;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int c = r[i >> 1][(i & 1) * 2 + w];
      o[2 * w] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, f, false));
      o[2 * w + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, f, true));
    }
    return o;
  }
};

// acc[weight row][column] += A B over the k values of one 16-byte piece of each lane
template <int EL>
__device__ __forceinline__ f32x4_t mma(i32x4_t a, i32x4_t b, f32x4_t acc) {
  if constexpr (EL == EL_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(a[i]), __int_as_float(b[i]), acc, 0, 0, 0);
    return acc;
  } else if constexpr (EL == EL_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), acc, 0,
                                                  0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   acc, 0, 0, 0);
  }
}

template <int EL>
__device__ __forceinline__ float load_one(const char *p, int64_t i) {
  if constexpr (EL == EL_F32) return ((const float *)p)[i];
  else return h16_to_f32<EL == EL_F16>(((const uint16_t *)p)[i]);
}

template <int EL>
__device__ __forceinline__ float bias_at(const MoeWeight &m, int e, int64_t r) {
  const char *b = m.bias_ptrs ? m.bias_ptrs[e] : m.bias ? m.bias + (int64_t)e * m.rows * elem_bytes(EL) : nullptr;
  return b ? load_one<EL>(b, r) : 0.f;
}

template <int WEL>
__device__ __forceinline__ int64_t row_bytes(int64_t cols) { return WEL == EL_MX ? cols : cols * elem_bytes(WEL); }

// First row r of expert e's matrix, and of its scales.
template <int WEL>
__device__ __forceinline__ const char *weight_row(const MoeWeight &m, int e, int64_t r) {
  const int64_t b = row_bytes<WEL>(m.cols);
  return (m.w_ptrs ? m.w_ptrs[e] : m.w + (int64_t)e * m.rows * b) + r * b;
}
__device__ __forceinline__ const uint8_t *scale_row(const MoeWeight &m, int e, int64_t r) {
  const int64_t b = m.cols / 32;
  return (m.scale_ptrs ? m.scale_ptrs[e] : m.scale + (int64_t)e * m.rows * b) + r * b;
}

// The tokens of the workgroup's expert, compacted in token order.
struct UpTokens {
  int expert, n;
  int slot[kMoeMaxTokens];    // first slot of the token that names the expert
  float gate[kMoeMaxTokens];  // the token's weight for it (all its slots that name it)
};

// Contraction over K for NT tiles of 16 columns and the gate's and up's rows.
template <int EL, int WEL, int NT, int U>
__device__ __forceinline__ void up_product(const MoeParams &p, const UpTokens &tok, int64_t f0, float *sums) {
  using W = Unit<WEL>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const uint32_t wb = (uint32_t)row_bytes<WEL>(p.K), xb = (uint32_t)(p.K * elem_bytes(EL));
  const int e = tok.expert;
  const auto wg = moe_rsrc(weight_row<WEL>(p.w1, e, f0)), wu = moe_rsrc(weight_row<WEL>(p.w1, e, p.F + f0));
  const auto sg = moe_rsrc(WEL == EL_MX ? scale_row(p.w1, e, f0) : nullptr);
  const auto su = moe_rsrc(WEL == EL_MX ? scale_row(p.w1, e, p.F + f0) : nullptr);
  const auto xr = moe_rsrc(p.x);
  const bool row_ok = f0 + col < p.F;
  const uint32_t end = row_ok ? wb : 0;  // past the last row: no byte is valid
  const uint32_t row = col * wb, srow = col * (uint32_t)(p.K / 32);
  uint32_t xrow[NT], xend[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + col;
    xend[t] = c < tok.n ? xb : 0;
    xrow[t] = c < tok.n ? (uint32_t)(tok.slot[c] / p.k) * xb : 0;
  }
  f32x4_t g[NT], u[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) g[t] = u[t] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  const int units = (int)((p.K + W::kElems - 1) / W::kElems);
  for (int c0 = wave; c0 < units; c0 += kUpWaves * U) {
    W ug[U], uu[U];
    i32x4_t b[U][NT][W::steps];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t c = c0 + i * kUpWaves;  // units past the end load zeros
      ug[i].load(wg, sg, row, c * 128, end, srow, q);
      uu[i].load(wu, su, row, c * 128, end, srow, q);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < W::steps; ++s) {
          const uint32_t at = c * W::b_bytes + W::b_byte(s, q);
          b[i][t][s] = load16(xr, at < xend[t] ? xrow[t] + at : kNowhere);
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int s = 0; s < W::steps; ++s) {
        const i32x4_t ag = ug[i].operand(s), au = uu[i].operand(s);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          g[t] = mma<EL>(ag, b[i][t][s], g[t]);
          u[t] = mma<EL>(au, b[i][t][s], u[t]);
        }
      }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float *o = sums + (((t * kUpWaves + wave) * 2) * 64 + lane) * 4;
    *(f32x4_t *)o = g[t];
    *(f32x4_t *)(o + 256) = u[t];
  }
}

// Rounds v to the weights' 16-bit type in two parts: v ~ hi + lo.
template <bool F16>
__device__ __forceinline__ void split(float v, uint16_t &hi, uint16_t &lo) {
  hi = f32_to_h16<F16>(v);
  const float rest = v - h16_to_f32<F16>(hi);
  lo = fabsf(rest) < INFINITY ? f32_to_h16<F16>(rest) : (uint16_t)0;  // hi is not finite
}

template <int EL, int WEL>
__global__ __launch_bounds__(kUpThreads) void moe_up_kernel(const MoeParams p) {
  __shared__ UpTokens tok;
  __shared__ __align__(16) float sums[4 * kUpWaves * 2 * 64 * 4];
  const int lane = threadIdx.x & 63;
  const int64_t f0 = (int64_t)blockIdx.x * kMoeRows;
  if (threadIdx.x < 64) {
    // lane t: the slots of token t that name the workgroup's expert
    const int e = p.E <= p.T * p.k ? (int)blockIdx.y : p.ids[blockIdx.y];
    int first = -1;
    float gate = 0.f;
    if (lane < p.T && e >= 0 && e < p.E)
#pragma unroll 4
      for (int j = 0; j < p.k; ++j) {
        const int s = lane * p.k + j;
        const float w = p.gates[s];
        if (p.ids[s] == e && w != 0.f) {
          if (first < 0) first = s;
          gate += w;
        }
      }
    const uint64_t mask = __ballot(first >= 0);
    const int rank = __popcll(mask & ((1ull << lane) - 1));
    if (first >= 0) {
      tok.slot[rank] = first;
      tok.gate[rank] = gate;
    }
    // one workgroup of several for the same expert goes on: the one of its first slot
    const int lead = mask ? __shfl(first, __ffsll((unsigned long long)mask) - 1) : -1;
    const bool mine = mask && (p.E <= p.T * p.k || lead == (int)blockIdx.y);
    if (lane == 0) {
      tok.expert = mine ? e : -1;
      tok.n = __popcll(mask);
    }
    if (blockIdx.x == 0) {
      if (lane == 0) p.entries[blockIdx.y] = {mine ? e : -1, 0, mask};
      p.slot_of[blockIdx.y * 64 + lane] = (int16_t)first;
    }
  }
  __syncthreads();
  if (tok.expert < 0) return;
  if (tok.n <= 16) up_product<EL, WEL, 1, WEL == EL_MX ? 2 : 4>(p, tok, f0, sums);
  else if (tok.n <= 32) up_product<EL, WEL, 2, WEL == EL_MX ? 1 : 2>(p, tok, f0, sums);
  else up_product<EL, WEL, 4, 1>(p, tok, f0, sums);
  __syncthreads();
  const int e = tok.expert, f = threadIdx.x & 15;
  if (f0 + f >= p.F) return;
  const float bg = bias_at<EL>(p.w1, e, f0 + f), bu = bias_at<EL>(p.w1, e, p.F + f0 + f);
  for (int c = threadIdx.x >> 4; c < tok.n; c += 16) {
    // row f, column c of a 16 x 16 result is value f % 4 of lane 16 (f / 4) + c % 16
    const float *s = sums + ((c >> 4) * kUpWaves * 2 * 64 + ((f >> 2) * 16 + (c & 15))) * 4 + (f & 3);
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < kUpWaves; ++w) {
      g += s[w * 512];
      u += s[w * 512 + 256];
    }
    g += bg;
    u += bu;
    const float a = tok.gate[c] * (g * sigmoid(g) * u);
    const int64_t at = tok.slot[c] * p.F + f0 + f;
    if constexpr (EL == EL_F32) {
      ((float *)p.a)[at] = a;
    } else {
      uint16_t *hi = (uint16_t *)p.a, *lo = hi + (int64_t)p.T * p.k * p.F;
      split<EL == EL_F16>(a, hi[at], lo[at]);
    }
  }
}

// LDS of the down kernel: the entries with an expert, in order.
struct DownEntry {
  uint64_t tokens;
  int32_t expert;
  int32_t base;  // its tokens' slots are slots[base ...]
};

template <int EL, int WEL, int NT, int U>
__global__ __launch_bounds__(kDownThreads) void moe_down_kernel(const MoeParams p) {
  using W = Unit<WEL>;
  extern __shared__ __align__(16) char lds[];
  __shared__ int wave_n[kDownWaves], wave_m[kDownWaves];
  float *sums = (float *)lds;  // at the end, over the table
  DownEntry *ent = (DownEntry *)lds;
  int16_t *slots = (int16_t *)(ent + p.n_entries);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kMoeRows;
  // compact the table: running counts of entries and of their tokens
  int n = 0, members = 0;
  for (int d0 = 0; d0 < p.n_entries; d0 += kDownThreads) {
    const int d = d0 + threadIdx.x;
    MoeEntry t{-1, 0, 0};
    if (d < p.n_entries) t = p.entries[d];
    const bool on = t.expert >= 0;
    const int mine = on ? __popcll(t.tokens) : 0;
    const uint64_t ons = __ballot(on);
    int upto = mine;  // inclusive sum over the wave's lanes
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(upto, s);
      if (lane >= s) upto += o;
    }
    if (lane == 63) {
      wave_n[wave] = __popcll(ons);
      wave_m[wave] = upto;
    }
    __syncthreads();
    int at = n + __popcll(ons & ((1ull << lane) - 1)), base = members + upto - mine;
    for (int w = 0; w < kDownWaves; ++w) {
      if (w < wave) {
        at += wave_n[w];
        base += wave_m[w];
      }
      n += wave_n[w];
      members += wave_m[w];
    }
    if (on) {
      ent[at] = {t.tokens, t.expert, base};
      uint64_t left = t.tokens;
      for (int i = base; left; ++i, left &= left - 1)
        slots[i] = p.slot_of[d * 64 + __ffsll((unsigned long long)left) - 1];
    }
    __syncthreads();
  }

  const uint32_t wb = (uint32_t)row_bytes<WEL>(p.F), ab = (uint32_t)(p.F * elem_bytes(EL));
  const uint32_t end = n0 + col < p.N ? wb : 0;
  const uint32_t row = col * wb, srow = col * (uint32_t)(p.F / 32);
  const auto ar = moe_rsrc(p.a);
  const auto lr = moe_rsrc(p.a + (int64_t)p.T * p.k * ab);
  f32x4_t acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  // items (entry, U units of F), dealt to the waves in turn
  const int pieces = (int)((p.F + W::kElems * U - 1) / (W::kElems * U));
  int i = wave / pieces, c = wave - i * pieces;
  W cur[U], nxt[U];
  const auto load = [&](W *w, int i, int c) {
    const int e = __builtin_amdgcn_readfirstlane(ent[i].expert);
    const auto r = moe_rsrc(weight_row<WEL>(p.w2, e, n0));
    const auto s = moe_rsrc(WEL == EL_MX ? scale_row(p.w2, e, n0) : nullptr);
#pragma unroll
    for (int j = 0; j < U; ++j) w[j].load(r, s, row, (c * U + j) * 128, end, srow, q);
  };
  if (i < n) load(cur, i, c);
  while (i < n) {
    int ni = i, nc = c + kDownWaves;
    while (nc >= pieces) {
      nc -= pieces;
      ++ni;
    }
    i32x4_t hi[NT][U * W::steps], lo[NT][U * W::steps];
    const uint64_t tokens = ent[i].tokens;
    const int base = ent[i].base;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int token = t * 16 + col;
      const bool on = (tokens >> token) & 1;
      const uint32_t arow =
          on ? (uint32_t)slots[base + __popcll(tokens & ((1ull << token) - 1))] * ab : 0;
      const uint32_t aend = on ? ab : 0;
#pragma unroll
      for (int s = 0; s < U * W::steps; ++s) {
        const uint32_t at = (c * U + s / W::steps) * W::b_bytes + W::b_byte(s % W::steps, q);
        const uint32_t off = at < aend ? arow + at : kNowhere;
        hi[t][s] = load16(ar, off);
        if constexpr (EL != EL_F32) lo[t][s] = load16(lr, off);
      }
    }
    if (ni < n) load(nxt, ni, nc);
    f32x4_t sum[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) sum[t] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < U * W::steps; ++s) {
      const i32x4_t a = cur[s / W::steps].operand(s % W::steps);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        sum[t] = mma<EL>(a, hi[t][s], sum[t]);
        if constexpr (EL != EL_F32) sum[t] = mma<EL>(a, lo[t][s], sum[t]);
      }
    }
    // only tokens that name the expert: an infinite weight times the zeros of another
    // token's column is NaN
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if ((tokens >> (t * 16 + col)) & 1) acc[t] += sum[t];
#pragma unroll
    for (int j = 0; j < U; ++j) cur[j] = nxt[j];
    i = ni;
    c = nc;
  }
  __syncthreads();  // every wave is done with the table
#pragma unroll
  for (int t = 0; t < NT; ++t) *(f32x4_t *)(sums + ((t * kDownWaves + wave) * 64 + lane) * 4) = acc[t];
  __syncthreads();
  const int r = threadIdx.x & 15;
  if (n0 + r >= p.N) return;
  for (int t = threadIdx.x >> 4; t < p.T; t += kDownThreads / 16) {
    const float *s = sums + ((t >> 4) * kDownWaves * 64 + ((r >> 2) * 16 + (t & 15))) * 4 + (r & 3);
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) y += s[w * 256];
    if (p.w2.bias || p.w2.bias_ptrs)
      for (int j = 0; j < p.k; ++j) {
        const int e = p.ids[t * p.k + j];
        const float w = p.gates[t * p.k + j];
        if (e >= 0 && e < p.E && w != 0.f) y = fmaf(w, bias_at<EL>(p.w2, e, n0 + r), y);
      }
    const int64_t at = t * p.N + n0 + r;
    if (p.residual) y += load_one<EL>(p.residual, at);
    if constexpr (EL == EL_F32) ((float *)p.y)[at] = y;
    else ((uint16_t *)p.y)[at] = f32_to_h16<EL == EL_F16>(y);
  }
}

size_t moe_workspace_bytes(int64_t T, int k, int E, int64_t F) {
  return moe_table_bytes((int)min64(T * k, E)) + (size_t)T * k * F * 4;
}

template <int EL, int WEL>
static void launch_moe_typed(const MoeParams &p, hipStream_t s) {
  hipLaunchKernelGGL((moe_up_kernel<EL, WEL>), dim3((unsigned)((p.F + kMoeRows - 1) / kMoeRows), p.n_entries),
                     dim3(kUpThreads), 0, s, p);
  const dim3 grid((unsigned)((p.N + kMoeRows - 1) / kMoeRows)), block(kDownThreads);
  const size_t table = (size_t)p.n_entries * sizeof(DownEntry) + (size_t)p.T * p.k * 2;  // at most 36 KiB
  const auto lds = [&](int tiles) {
    const size_t sums = (size_t)tiles * kDownWaves * 64 * 16;
    return table > sums ? (table + 15) & ~(size_t)15 : sums;
  };
  if (p.T <= 16)
    hipLaunchKernelGGL((moe_down_kernel<EL, WEL, 1, WEL == EL_MX ? 1 : 2>), grid, block, lds(1), s, p);
  else if (p.T <= 32)
    hipLaunchKernelGGL((moe_down_kernel<EL, WEL, 2, 1>), grid, block, lds(2), s, p);
  else
    hipLaunchKernelGGL((moe_down_kernel<EL, WEL, 4, 1>), grid, block, lds(4), s, p);
}

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
  p.T = (int)T;
  p.k = k;
  p.E = E;
  p.K = K;
  p.F = F;
  p.N = N;
  p.n_entries = (int)min64(T * k, E);
  p.entries = (MoeEntry *)ws;
  p.slot_of = (int16_t *)(p.entries + p.n_entries);
  p.a = (char *)ws + moe_table_bytes(p.n_entries);
  if (mx) launch_moe_typed<EL_BF16, EL_MX>(p, s);
  else if (el == EL_F32) launch_moe_typed<EL_F32, EL_F32>(p, s);
  else if (el == EL_F16) launch_moe_typed<EL_F16, EL_F16>(p, s);
  else launch_moe_typed<EL_BF16, EL_BF16>(p, s);
  return hipGetLastError();
}

}  // namespace gl
