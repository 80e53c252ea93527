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
//   down  workgroup (16 columns of y): its waves share the (expert, piece of F) items of
//         the whole call, an item's columns being the expert's tokens again; each wave
//         adds its products to its own sum of every token in LDS, and the waves' sums are
//         added at the end: no atomics, a fixed order.
//
// For 16-bit weights a is kept as two values of the weights' type, the rounded value and
// the rest, each multiplied in its own MFMA step: the products see 16 significant bits
// of a (22 for fp16) where one value would add its own rounding, of the output's size,
// to the result.  The extra step is free beside the weight read.
#include <type_traits>

#include "gl_vec.hpp"

namespace gl {

enum { EL_MX = 3 };  // weights: E4M3 codes with an E8M0 scale per 32 of a row
constexpr int kMoeMaxTokens = 64;
constexpr int kUpThreads = 256, kUpWaves = kUpThreads / 64;
// Units that a wave takes at a time (an MXFP8 unit holds twice the k values).
template <int WEL>
constexpr int up_units() { return WEL == EL_MX ? 1 : 2; }
template <int WEL>
constexpr int down_units() { return WEL == EL_MX ? 2 : 4; }
constexpr int kDownThreads = 512, kDownWaves = kDownThreads / 64;
constexpr int kMoeRows = 16;  // weight rows of a workgroup (per half of W1)

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
  uint64_t tokens;  // bit t: token t has a slot of it
  int32_t expert;   // -1: none
  int32_t first;    // slot_of its first token
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
                       uint32_t, bool, int q) {
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
  uint32_t s;  // the 4 scales of the unit's codes in the lane's row
  int q;
  __device__ static uint32_t b_byte(int i, int q) { return (i >> 1) * 128 + q * 32 + (i & 1) * 16; }
  __device__ void load(__amdgpu_buffer_rsrc_t w, __amdgpu_buffer_rsrc_t sc, uint32_t row, uint32_t at, uint32_t end,
                       uint32_t srow, bool wide, int q_) {
    q = q_;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t b = at + i * 64 + q * 16;
      r[i] = load16(w, b < end ? row + b : kNowhere);
    }
    // whole units (wide): their 4 scales are an aligned word
    if (wide) {
      s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(sc, (int)(at < end ? srow + at / 32 : kNowhere), 0, 0);
      return;
    }
    s = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t b = at + i * 64 + q * 16;
      const uint32_t v = __builtin_amdgcn_raw_buffer_load_b8(sc, (int)(b < end ? srow + b / 32 : kNowhere), 0, 0);
      s |= (v & 0xff) << (16 * i + 8 * (q >> 1));
    }
  }
  // 8 codes as bf16: their values are exact there.  The conversion takes the exponent
  // field of an fp32 scale, which is the E8M0 byte (255, NaN, included).
  __device__ i32x4_t operand(int i) const {
    const uint32_t byte = (s >> (16 * (i >> 1) + 8 * (q >> 1))) & 0xff;
    const float f = __uint_as_float(byte << 23);
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

// The weight side of the up kernel: units wave, wave + kUpWaves, ... of the gate's and the
// up's 16 rows, U of each at a time.
template <int WEL>
struct UpWeights {
  static constexpr int U = up_units<WEL>();
  using W = Unit<WEL>;
  __amdgpu_buffer_rsrc_t wg, wu, sg, su;
  uint32_t row, srow, end;
  int q;
  bool wide;
  __device__ UpWeights(const MoeParams &p, int e, int64_t f0) {
    const int col = threadIdx.x & 15;
    const uint32_t wb = (uint32_t)row_bytes<WEL>(p.K);
    wg = moe_rsrc(weight_row<WEL>(p.w1, e, f0));
    wu = moe_rsrc(weight_row<WEL>(p.w1, e, p.F + f0));
    sg = moe_rsrc(WEL == EL_MX ? scale_row(p.w1, e, f0) : nullptr);
    su = moe_rsrc(WEL == EL_MX ? scale_row(p.w1, e, p.F + f0) : nullptr);
    q = (threadIdx.x >> 4) & 3;
    row = col * wb;
    wide = p.K % 128 == 0;
    srow = col * (uint32_t)(p.K / 32);
    end = f0 + col < p.F ? wb : 0;  // past the last row: no byte is valid
  }
  // units past the end load zeros
  __device__ void load(W *g, W *u, int c0) const {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t at = (uint32_t)(c0 + i * kUpWaves) * 128;
      g[i].load(wg, sg, row, at, end, srow, wide, q);
      u[i].load(wu, su, row, at, end, srow, wide, q);
    }
  }
};

// Contraction over K for up to NT tiles of 16 columns; g and u hold the first units.
template <int EL, int WEL, int NT>
__device__ __forceinline__ void up_product(const MoeParams &p, const UpTokens &tok, const UpWeights<WEL> &weights,
                                           Unit<WEL> *g, Unit<WEL> *u, float *sums) {
  using W = Unit<WEL>;
  constexpr int U = up_units<WEL>();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const uint32_t xb = (uint32_t)(p.K * elem_bytes(EL));
  const auto xr = moe_rsrc(p.x);
  uint32_t xrow[NT], xend[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + col;
    xend[t] = c < tok.n ? xb : 0;
    xrow[t] = c < tok.n ? (uint32_t)(tok.slot[c] / p.k) * xb : 0;
  }
  f32x4_t ag[NT], au[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) ag[t] = au[t] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  const int units = (int)((p.K + W::kElems - 1) / W::kElems);
  const auto step = [&](int c0, const W *g, const W *u, W *ng, W *nu) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t && t * 16 >= tok.n) break;
      // the tokens' pieces come from cache, the next weights from memory: issued in this
      // order, the products wait for the former alone
      i32x4_t b[U][W::steps];
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int s = 0; s < W::steps; ++s) {
          const uint32_t at = (uint32_t)(c0 + i * kUpWaves) * W::b_bytes + W::b_byte(s, q);
          b[i][s] = load16(xr, at < xend[t] ? xrow[t] + at : kNowhere);
        }
      if (t == 0) weights.load(ng, nu, c0 + kUpWaves * U);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int s = 0; s < W::steps; ++s) {
          ag[t] = mma<EL>(g[i].operand(s), b[i][s], ag[t]);
          au[t] = mma<EL>(u[i].operand(s), b[i][s], au[t]);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // two register sets in turn: copying one to the other would wait for its loads
  W ng[U], nu[U];
  for (int c0 = wave; c0 < units; c0 += 2 * kUpWaves * U) {
    step(c0, g, u, ng, nu);
    if (c0 + kUpWaves * U >= units) break;
    step(c0 + kUpWaves * U, ng, nu, g, u);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float *o = sums + (((t * kUpWaves + wave) * 2) * 64 + lane) * 4;
    *(f32x4_t *)o = ag[t];
    *(f32x4_t *)(o + 256) = au[t];
  }
}

// Rounds v to the weights' 16-bit type in two parts: v ~ hi + lo.
template <bool F16>
__device__ __forceinline__ void split(float v, uint16_t &hi, uint16_t &lo) {
  hi = f32_to_h16<F16>(v);
  const float rest = v - h16_to_f32<F16>(hi);
  lo = fabsf(rest) < INFINITY ? f32_to_h16<F16>(rest) : (uint16_t)0;  // hi is not finite
}

template <int EL, int WEL, int NT>
__global__ __launch_bounds__(kUpThreads) void moe_up_kernel(const MoeParams p) {
  __shared__ UpTokens tok;
  __shared__ __align__(16) float sums[NT * kUpWaves * 2 * 64 * 4];
  const int lane = threadIdx.x & 63;
  const int64_t f0 = (int64_t)blockIdx.x * kMoeRows;
  const bool by_expert = p.E <= p.T * p.k;
  const int e = by_expert ? (int)blockIdx.y : p.ids[blockIdx.y];
  const bool valid = e >= 0 && e < p.E;
  // lane t of the first wave: the slots of token t, 8 at a time, loaded ahead of the weights
  const bool search = threadIdx.x < 64 && lane < p.T && valid;
  int id[8];
  float w[8];
  const auto slots = [&](int j0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = lane * p.k + (j0 + i < p.k ? j0 + i : j0);
      id[i] = p.ids[s];
      w[i] = p.gates[s];
    }
  };
  if (search) slots(0);
  const UpWeights<WEL> weights(p, valid ? e : 0, f0);
  Unit<WEL> g[up_units<WEL>()], u[up_units<WEL>()];
  // a slot's expert is almost always read: its first weights are on their way during the
  // search for its tokens
  if (valid && !by_expert) weights.load(g, u, threadIdx.x >> 6);
  if (threadIdx.x < 64) {
    // the slots of token t that name the workgroup's expert
    int first = -1;
    float gate = 0.f;
    if (search)
      for (int j0 = 0; j0 < p.k; j0 += 8) {
        if (j0) slots(j0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j0 + i < p.k && id[i] == e && w[i] != 0.f) {
            if (first < 0) first = lane * p.k + j0 + i;
            gate += w[i];
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
    const bool mine = mask && (by_expert || lead == (int)blockIdx.y);
    if (lane == 0) {
      tok.expert = mine ? e : -1;
      tok.n = __popcll(mask);
    }
    if (blockIdx.x == 0) {
      if (lane == 0) p.entries[blockIdx.y] = {mask, mine ? e : -1, lead};
      p.slot_of[blockIdx.y * 64 + lane] = (int16_t)first;
    }
  }
  __syncthreads();
  if (tok.expert < 0) return;
  if (by_expert) weights.load(g, u, threadIdx.x >> 6);
  up_product<EL, WEL, NT>(p, tok, weights, g, u, sums);
  __syncthreads();
  const int f = threadIdx.x & 15;
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
  int32_t expert;
  int32_t base, n;  // its tokens' slots are slots[base ... base + n)
};

template <int EL, int WEL, int R>
__global__ __launch_bounds__(kDownThreads) void moe_down_kernel(const MoeParams p) {
  using W = Unit<WEL>;
  constexpr int U = down_units<WEL>();
  extern __shared__ __align__(16) char lds[];
  __shared__ int wave_n[kDownWaves], wave_m[kDownWaves];
  float *acc = (float *)lds;  // [waves][T][16 rows] sums of a token
  DownEntry *ent = (DownEntry *)(acc + kDownWaves * p.T * 16);
  int16_t *slots = (int16_t *)(ent + p.n_entries);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * R;
  for (int i = threadIdx.x; i < kDownWaves * p.T * 4; i += kDownThreads) ((f32x4_t *)acc)[i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  // compact the table: running counts of entries and of their tokens
  int n = 0, members = 0;
  for (int d0 = 0; d0 < p.n_entries; d0 += kDownThreads) {
    const int d = d0 + threadIdx.x;
    MoeEntry t{0, -1, 0};
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
      ent[at] = {t.expert, base, mine};
      slots[base] = (int16_t)t.first;
      uint64_t left = t.tokens & (t.tokens - 1);
      for (int i = base + 1; left; ++i, left &= left - 1)
        slots[i] = p.slot_of[d * 64 + __ffsll((unsigned long long)left) - 1];
    }
    __syncthreads();
  }

  const uint32_t wb = (uint32_t)row_bytes<WEL>(p.F), ab = (uint32_t)(p.F * elem_bytes(EL));
  const uint32_t end = col < R && n0 + col < p.N ? wb : 0;
  const uint32_t row = col * wb, srow = col * (uint32_t)(p.F / 32);
  const bool wide = p.F % 128 == 0;
  const auto ar = moe_rsrc(p.a);
  constexpr int kCols = EL == EL_F32 ? 16 : 8;  // tokens of a step
  const int token = col & (kCols - 1);
  const uint32_t part = col < kCols ? 0 : (uint32_t)(p.T * p.k) * ab;  // the second parts' plane
  // items (entry, U units of F), dealt to the waves in turn
  const int pieces = (int)((p.F + W::kElems * U - 1) / (W::kElems * U));
  const auto load = [&](W *w, int i, int c) {
    const int e = __builtin_amdgcn_readfirstlane(ent[i].expert);
    const auto r = moe_rsrc(weight_row<WEL>(p.w2, e, n0));
    const auto s = moe_rsrc(WEL == EL_MX ? scale_row(p.w2, e, n0) : nullptr);
#pragma unroll
    for (int j = 0; j < U; ++j) w[j].load(r, s, row, (c * U + j) * 128, end, srow, wide, q);
  };
  int i = wave / pieces, c = wave - i * pieces;
  // one item with its weights in `cur`; moves on to the next, whose weights go to `nxt`
  const auto step = [&](const W *cur, W *nxt) {
    int ni = i, nc = c + kDownWaves;
    while (nc >= pieces) {
      nc -= pieces;
      ++ni;
    }
    const int base = __builtin_amdgcn_readfirstlane(ent[i].base), m = __builtin_amdgcn_readfirstlane(ent[i].n);
    // the entry's tokens as columns; a 16-bit a's two parts are columns of the same step
    for (int t = 0; t < m; t += kCols) {
      const bool on = t + token < m;
      const int slot = on ? slots[base + t + token] : 0;
      const uint32_t arow = (uint32_t)slot * ab + part, aend = on ? ab : 0;
      i32x4_t b[U * W::steps];
#pragma unroll
      for (int s = 0; s < U * W::steps; ++s) {
        const uint32_t at = (c * U + s / W::steps) * W::b_bytes + W::b_byte(s % W::steps, q);
        b[s] = load16(ar, at < aend ? arow + at : kNowhere);
      }
      if (t == 0 && ni < n) load(nxt, ni, nc);
      __builtin_amdgcn_sched_barrier(0);
      f32x4_t sum = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < U * W::steps; ++s) sum = mma<EL>(cur[s / W::steps].operand(s % W::steps), b[s], sum);
      if constexpr (kCols == 8)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] += __shfl_xor(sum[r], 8);
      if (on && col == token) {  // each column another token: no lane shares a sum
        f32x4_t *o = (f32x4_t *)(acc + (wave * p.T + slot / p.k) * 16 + q * 4);
        *o += sum;
      }
    }
    i = ni;
    c = nc;
  };
  // two register sets in turn: copying one to the other would wait for its loads
  W w0[U], w1[U];
  if (i < n) load(w0, i, c);
  while (i < n) {
    step(w0, w1);
    if (i >= n) break;
    step(w1, w0);
  }
  __syncthreads();
  for (int o = threadIdx.x; o < p.T * 16; o += kDownThreads) {
    const int r = o & 15, t = o >> 4;
    if (r >= R || n0 + r >= p.N) continue;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) y += acc[w * p.T * 16 + o];
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
  const dim3 up((unsigned)((p.F + kMoeRows - 1) / kMoeRows), p.n_entries);
  if (p.T <= 16)
    hipLaunchKernelGGL((moe_up_kernel<EL, WEL, 1>), up, dim3(kUpThreads), 0, s, p);
  else
    hipLaunchKernelGGL((moe_up_kernel<EL, WEL, 4>), up, dim3(kUpThreads), 0, s, p);
  // LDS: at most 4 KiB of sums a wave, 24 KiB of entries and 4 KiB of slots
  const size_t lds = (size_t)kDownWaves * p.T * 64 + (size_t)p.n_entries * sizeof(DownEntry) + (size_t)p.T * p.k * 2;
  if (p.N / 16 < 256)
    hipLaunchKernelGGL((moe_down_kernel<EL, WEL, 8>), dim3((unsigned)((p.N + 7) / 8)), dim3(kDownThreads), lds, s, p);
  else
    hipLaunchKernelGGL((moe_down_kernel<EL, WEL, 16>), dim3((unsigned)((p.N + 15) / 16)), dim3(kDownThreads), lds, s,
                       p);
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
