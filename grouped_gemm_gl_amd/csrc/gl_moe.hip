// The expert layer for a few tokens: for token t with experts e_j = ids[t, j] and
// weights w_j
//   y_t = residual_t + sum_j w_j (W2_e SwiGLU(W1_e x_t + b1_e) + b2_e)
// in two kernels, without sorting or gathering rows.  A slot whose id is no expert of
// this call, or whose weight is 0, takes no part.
//
// Both are bound by reading the used experts' weights once from HBM, and what a load
// instruction touches decides how near they come: one that takes 16 rows by 64 bytes, the
// layout of the MFMA's operand, streams 4.2 TB/s where one that takes 1 KiB of a row streams
// 5.9 (67 MB over 512 workgroups; 16 rows of 8 would cost the same again).  So every weight
// goes straight from memory to the registers of the one wave that uses it, no load takes less
// than whole 128-byte lines, and the next loads are in flight during the products (but for the
// W2 kernel's MFMA steps, see down_many):
//
//   - experts of many tokens by MFMA steps of 16 weight rows by 16 columns, the columns being
//     the expert's tokens, compacted; loads of 8 rows by 128 bytes and a rotation of 8 lanes
//     give the operand's layout (RowPair);
//   - experts of one or two tokens (up to four) by dot products in the lane over 1 KiB blocks
//     of 8 rows, the lanes' sums added at the end (vec_sum).
//
//   up    workgroup (expert, 16 columns of a): its waves split the contraction over K and add
//         up through LDS, or, by dot products, take 4 columns each (8 a workgroup where all
//         go that way).  Leaves
//         a = w SwiGLU(W1 x + b1), w the token's weight for the expert, in the workspace.
//   down  workgroup (16 or 8 columns of y): its waves share the (expert, piece of F) items of
//         the whole call; each wave adds its products to its own sum of every token in LDS,
//         and the waves' sums are added at the end: no atomics, a fixed order.
//
// Between the kernels a is fp32 beside fp32 and fp16 weights, and for bf16 products two bf16
// values, the rounded value and the rest (2^-18 of a or less is lost).  An MFMA step of 16-bit
// weights takes a as two such parts, which share the step as two columns: the products see at
// least 16 significant bits of a where one value would add its own rounding, of the output's
// size, to the result.  (With bf16 parts 0.2-0.5% of the outputs round to the other neighbour of
// the exact value, in an fp32 computation 0.1%; the error against 64 bits, 1.66e-3 of the norm,
// is the same to six digits.  A third part would leave a step five tokens instead of eight.)
// fp16's exponents are too few for that (a = 70000 is no fp16 value, and
// of 1e-5 the two parts would keep 8 bits), so the fp16 parts are made in the down kernel under
// a power-of-two scale for a token's 256 columns of an item (ScaledColumns): 2^-20 of a value
// or 2^-49 of the largest of the 256 is lost, over fp32's whole range.  Its dot products take
// the fp32 values as they are.
//
// Measured (kernel times): 64 tokens over 256 experts of 7168/2048, bf16: up 1.85 ms (7.0
// TB/s of weights), down 1.11 ms (5.9 TB/s: 448 workgroups over 256 CUs); one token, 8 of 64
// experts of 2048/768: up 12.7 us, down 9.0 us, half of it latency.
#include <type_traits>

#include "gl_vec.hpp"

namespace gl {

// Weights as E4M3 codes with an E8M0 scale per 32 of a row; EL_MX: K and F are multiples of
// 128 above 128, so that a row has eight scales from an aligned word on, EL_MX_RAGGED: of 32.
enum { EL_MX = 3, EL_MX_RAGGED = 4 };
typedef __attribute__((ext_vector_type(2))) int i32x2_t;
constexpr bool is_mx(int wel) { return wel >= EL_MX; }
constexpr int kMoeMaxTokens = 64, kCUs = 256;
constexpr int kUpThreads = 256, kUpWaves = kUpThreads / 64;
// Units that a wave takes at a time, in the up kernel (an MXFP8 unit holds twice the k values)
// and in the down kernel (MXFP8, 17 tokens over 32 experts of 4096/2048: 44.3 us, 2 units 46.2).
template <int WEL>
constexpr int up_units() { return is_mx(WEL) ? 1 : 2; }
constexpr int kDownUnits = 4;
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
  char *a;            // [T k][F] fp32, or two planes [T k][F] of bf16
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

// Weights are read once, whole lines at a time: non-temporal loads (the up kernel at 64
// tokens, 256 experts of 7168/2048, 13.1 GB: 1.83 ms, 2.04 without).
__device__ __forceinline__ i32x4_t load_weight(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 2));
}
__device__ __forceinline__ i32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

// 16 rows of an MFMA operand (weight rows, or the tokens that are its columns), 128 bytes
// of each: lane (r, q) = (l % 16, l / 16) needs two 16-byte chunks of row r, which the two
// loads would each take as 16 rows by 64 bytes.  Instead `low` takes rows 0-7 and `high`
// rows 8-15, whole 128-byte lines, the lanes of r and r + 8 sharing a row, and one rotation
// of 8 lanes a register gives either chunk to its lane.
struct RowPair {
  i32x4_t low, high;
  // chunk `h` (0 or 1) of the lane's row; the lanes r loaded theirs as chunk r / 8
  __device__ __forceinline__ i32x4_t chunk(int h) const {
    i32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // row_ror:8 into the lanes of rows 8-15, or 0-7
      o[i] = h == 0 ? __builtin_amdgcn_update_dpp(low[i], high[i], 0x128, 0xf, 0xc, false)
                    : __builtin_amdgcn_update_dpp(high[i], low[i], 0x128, 0xf, 0x3, false);
    return o;
  }
};

// Where the lane's weight rows are: offsets from the first of the workgroup's R rows.
struct WeightLane {
  uint32_t row, end_low, end_high, step, chunk;  // step: from row r to r + 8
  uint32_t srow, send, wb;                       // scales of row l % 16
  int q;
  // rows: how many of the 16 there are; wb: bytes of one
  __device__ WeightLane(int64_t rows, uint32_t wb, int64_t cols) : wb(wb) {
    const int lane = threadIdx.x & 63, r = lane & 15;
    q = lane >> 4;
    row = (r & 7) * wb;
    step = 8 * wb;
    end_low = (r & 7) < rows ? wb : 0;  // past the last row no byte is valid
    end_high = (r & 7) + 8 < rows ? wb : 0;
    chunk = (r >> 3) * 64 + q * 16;
    srow = r * (uint32_t)(cols / 32);
    send = r < rows ? wb : 0;
  }
};

// A unit is 128 bytes of each of R = 16 or 8 weight rows; its k values are taken in the
// order that the lanes' chunks give, the same for both operands, in `steps` pieces: piece i
// contracts the 16 bytes that b_byte(i) names of each token's row.
template <int WEL, int R>
struct Unit {  // bf16, fp16 and fp32 weights
  static constexpr int kElems = 128 / elem_bytes(WEL);
  static constexpr int steps = 2;
  static constexpr bool pairs = false;
  static constexpr int b_bytes = 128;  // of a token's row
  RowPair r;
  __device__ static uint32_t b_byte(int i, int q) { return i * 64 + q * 16; }
  __device__ void load(__amdgpu_buffer_rsrc_t w, __amdgpu_buffer_rsrc_t, const WeightLane &o, uint32_t at) {
    const uint32_t b = at + o.chunk;
    r.low = load_weight(w, b < o.end_low ? o.row + b : kNowhere);
    r.high = (i32x4_t){0, 0, 0, 0};
    if constexpr (R == 16) r.high = load_weight(w, b < o.end_high ? o.row + o.step + b : kNowhere);
  }
  __device__ void load_scales(__amdgpu_buffer_rsrc_t, const WeightLane &, uint32_t) {}
  __device__ void take_scales(const WeightLane &, uint32_t, Unit &) {}
  __device__ i32x4_t operand(int i) const { return r.chunk(i); }
};

template <int WEL, int R>
struct CodeUnit {  // MXFP8 weights
  static constexpr int kElems = 128;
  static constexpr int steps = 4;
  static constexpr int b_bytes = 256;
  // A load of scales touches 16 lines, one of codes 8: two units' scales are one load.
  static constexpr bool pairs = WEL == EL_MX;
  RowPair r;
  uint32_t s;  // the 4 scales of the unit's codes in row l % 16
  i32x2_t s2;  // with `pairs`: of this and the next unit, as loaded
  int q;
  __device__ static uint32_t b_byte(int i, int q) { return (i >> 1) * 128 + q * 32 + (i & 1) * 16; }
  __device__ void load(__amdgpu_buffer_rsrc_t w, __amdgpu_buffer_rsrc_t sc, const WeightLane &o, uint32_t at) {
    q = o.q;
    const uint32_t b = at + o.chunk;
    r.low = load_weight(w, b < o.end_low ? o.row + b : kNowhere);
    r.high = (i32x4_t){0, 0, 0, 0};
    if constexpr (R == 16) r.high = load_weight(w, b < o.end_high ? o.row + o.step + b : kNowhere);
    if constexpr (pairs) return;
    s = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t c = at + i * 64 + q * 16;
      const uint32_t v = __builtin_amdgcn_raw_buffer_load_b8(sc, (int)(c < o.send ? o.srow + c / 32 : kNowhere), 0, 0);
      s |= (v & 0xff) << (16 * i + 8 * (q >> 1));
    }
  }
  // Scales of the units at `at` and behind it; where the former is the row's last, of it and
  // the one before (a row has two units or more).
  __device__ void load_scales(__amdgpu_buffer_rsrc_t sc, const WeightLane &o, uint32_t at) {
    const uint32_t from = at / 32 - (at + 128 >= o.wb ? 4 : 0);
    s2 = __builtin_bit_cast(
        i32x2_t, __builtin_amdgcn_raw_buffer_load_b64(sc, (int)(at < o.send ? o.srow + from : kNowhere), 0, 0));
  }
  // Takes its scales, and gives the next unit its own, when the load is waited for.
  __device__ void take_scales(const WeightLane &o, uint32_t at, CodeUnit &next) {
    const bool last = at + 128 >= o.wb;
    s = (uint32_t)(last ? s2[1] : s2[0]);
    next.s = last ? 0u : (uint32_t)s2[1];
  }
  // 8 codes as bf16: their values are exact there.  The conversion takes the exponent
  // field of an fp32 scale, which is the E8M0 byte (255, NaN, included).
  __device__ i32x4_t operand(int i) const {
    const uint32_t byte = (s >> (16 * (i >> 1) + 8 * (q >> 1))) & 0xff;
    const float f = __uint_as_float(byte << 23);
    const i32x4_t codes = r.chunk(i >> 1);
    i32x4_t o;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int c = codes[(i & 1) * 2 + w];
      o[2 * w] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, f, false));
      o[2 * w + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, f, true));
    }
    return o;
  }
};

template <int R>
struct Unit<EL_MX, R> : CodeUnit<EL_MX, R> {};
template <int R>
struct Unit<EL_MX_RAGGED, R> : CodeUnit<EL_MX_RAGGED, R> {};

// The tokens' side of U units: pair j holds pieces 2 j and 2 j + 1 of the columns.
// row_low / row_high: byte offsets of the lane's rows among columns 0-7 and 8-15, each
// valid up to its end; HIGH: whether columns 8-15 hold any token.  (Decided here and not at
// run time: a branch around loads makes the compiler wait for those before it.)
template <class W, int U, bool HIGH>
struct Columns {
  RowPair b[U * W::steps / 2];
  __device__ void load(__amdgpu_buffer_rsrc_t x, uint32_t row_low, uint32_t end_low, uint32_t row_high,
                       uint32_t end_high, const uint32_t *unit_at) {
    const int lane = threadIdx.x & 63, h = (lane >> 3) & 1, q = lane >> 4;
#pragma unroll
    for (int j = 0; j < U * W::steps / 2; ++j) {
      const int i = (2 * j) % W::steps;  // piece of the unit
      const uint32_t at = unit_at[2 * j / W::steps] + (h ? W::b_byte(i + 1, q) : W::b_byte(i, q));
      b[j].low = load16(x, at < end_low ? row_low + at : kNowhere);
      b[j].high = (i32x4_t){0, 0, 0, 0};
      if constexpr (HIGH) b[j].high = load16(x, at < end_high ? row_high + at : kNowhere);
    }
  }
  __device__ i32x4_t operand(int piece) const { return b[piece / 2].chunk(piece & 1); }
};

// Rounds v to bf16 in two parts: v ~ hi + lo.
__device__ __forceinline__ void split(float v, uint16_t &hi, uint16_t &lo) {
  hi = f32_to_h16<false>(v);
  const float rest = v - h16_to_f32<false>(hi);
  lo = fabsf(rest) < INFINITY ? f32_to_h16<false>(rest) : (uint16_t)0;  // hi is not finite
}

// A sum of weights times a from those of a's two parts.  Where the leading one is not finite it
// tells all: an infinite weight meets the rest as NaN or in the other sign.
__device__ __forceinline__ float join(float leading, float rest) {
  return fabsf(leading) < INFINITY ? leading + rest : leading;
}

// The tokens' side of U units from fp32 values for fp16 products, two columns a token: the value's leading bits in
// columns 0-7 and the rest in 8-15, both in the scale 2^shift that brings the largest of the U
// units' values to 2^14 ... 2^15, the rest 2^11 above that.  (The weights' sums are divided by
// both afterwards.)  Both parts are cut off rather than rounded, which keeps them below 2^15.
// The lanes of a token's two columns each load and split half of the 8 values that both need,
// so a load takes whole lines (8 rows by 128 bytes: 64 tokens over 8 experts of 4096/14336 take
// 704 us, 711 where each lane loads 32 bytes of its own), and change halves by rotations.  The
// splitting is some 150 instructions an item that its wave waits for (stored unscaled parts, as
// bf16's are, took 695 us there, but hold neither 70000 nor 16 bits of 10^-3).
constexpr float kRestScale = 2048.f;
template <class W, int U>
struct ScaledColumns {
  static constexpr int n = U * W::steps;
  i32x4_t b[n];  // 4 fp32 values of a piece; split: two words of leading bits, two of the rest
  int shift;
  // row / end: the lane's token (l % 8) in bytes of fp32
  __device__ void load(__amdgpu_buffer_rsrc_t a, uint32_t row, uint32_t end, const uint32_t *unit_at) {
    const int lane = threadIdx.x & 63, h = (lane >> 3) & 1, q = lane >> 4;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const uint32_t at = 2 * (unit_at[j / W::steps] + W::b_byte(j % W::steps, q)) + 16 * h;
      b[j] = load16(a, at < end ? row + at : kNowhere);
    }
  }
  __device__ void split() {
    float top = 0.f;  // (NaN leaves it as it is)
#pragma unroll
    for (int j = 0; j < n; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(__int_as_float(b[j][i])));
    // over the token's eight lanes: l ^ 8 by a rotation, l ^ 16 and l ^ 32 by swaps
    top = fmaxf(top, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(top), 0x128, 0xf, 0xf, true)));
    const auto s16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(top), __float_as_uint(top), false, false);
    top = fmaxf(__uint_as_float(s16[0]), __uint_as_float(s16[1]));
    const auto s32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
    top = fmaxf(__uint_as_float(s32[0]), __uint_as_float(s32[1]));
    shift = min(141 - (int)(__float_as_uint(top) >> 23), 127);
    const float scale = __uint_as_float((uint32_t)(shift + 127) << 23);
#pragma unroll
    for (int j = 0; j < n; ++j) {
      i32x4_t o;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float v = __int_as_float(b[j][2 * i]) * scale, w = __int_as_float(b[j][2 * i + 1]) * scale;
        const auto h = __builtin_amdgcn_cvt_pkrtz(v, w);
        o[i] = __builtin_bit_cast(int, h);
        o[2 + i] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_pkrtz((v - (float)h[0]) * kRestScale,
                                                                      (w - (float)h[1]) * kRestScale));
      }
      b[j] = o;
    }
  }
  // lanes 0-7 of 16: their own leading bits, then those of l + 8; lanes 8-15: the rest of
  // l - 8, then their own
  __device__ i32x4_t operand(int piece) const {
    const i32x4_t v = b[piece];
    i32x4_t o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o[i] = __builtin_amdgcn_update_dpp(v[i], v[2 + i], 0x128, 0xf, 0xc, false);
      o[2 + i] = __builtin_amdgcn_update_dpp(v[2 + i], v[i], 0x128, 0xf, 0x3, false);
    }
    return o;
  }
  // a token's sum from those of its two columns (an infinite weight gives NaN where a is below
  // 2^-39 of the largest: its leading part is 0)
  __device__ float sum(float leading, float rest) const { return ldexpf(join(leading, rest * (1.f / kRestScale)), -shift); }
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
__device__ __forceinline__ int64_t row_bytes(int64_t cols) { return is_mx(WEL) ? cols : cols * elem_bytes(WEL); }

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

// ------------------------------------------------------------------ few columns --
// One wave takes 1 KiB blocks of 8 rows, 16 bytes of each row in a lane, and the tokens'
// values of the same places beside them.
constexpr int kVecRows = 8;

template <int WEL>
constexpr int block_elems() { return is_mx(WEL) ? 1024 : 1024 / elem_bytes(WEL); }

// The lane's 16 bytes of each of 8 rows.
template <int WEL>
struct VecRows {
  i32x4_t r[kVecRows];
  uint8_t s[is_mx(WEL) ? kVecRows : 1];
  // row byte offsets from the resource's base are i * wb; a row not < rows is not read
  __device__ void load(__amdgpu_buffer_rsrc_t w, __amdgpu_buffer_rsrc_t sc, int first, int n, uint32_t at, uint32_t wb,
                       int rows) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool ok = at < wb && i < rows;
      r[first + i] = load_weight(w, ok ? i * wb + at : kNowhere);
      if constexpr (is_mx(WEL))
        s[first + i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(sc, (int)(ok ? (i * wb + at) / 32 : kNowhere), 0, 0);
    }
  }
};

// A lane's values of one token at the places of its 16 weight bytes: 16 bytes of the
// activations' type, or 32 beside MXFP8 codes and where fp32 values meet fp16 weights.
template <int WEL, bool WIDE = is_mx(WEL)>
struct VecToken {
  static constexpr int parts = WIDE ? 2 : 1;
  i32x4_t v[parts];
  __device__ void load(__amdgpu_buffer_rsrc_t x, uint32_t row, uint32_t at, uint32_t xb) {
#pragma unroll
    for (int i = 0; i < parts; ++i) v[i] = load16(x, at + 16 * i < xb ? row + at + 16 * i : kNowhere);
  }
};

template <int EL>
__device__ __forceinline__ float dot2(int a, int b, float c) {
  if constexpr (EL == EL_F16) {
    typedef __attribute__((ext_vector_type(2))) _Float16 h2;
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b), c, false);
  } else {
    typedef __attribute__((ext_vector_type(2))) __bf16 b2;
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, a), __builtin_bit_cast(b2, b), c, false);
  }
}

// acc[r][c P + d] += row r . part d of token c over the lane's places, for n tokens
template <int EL, int WEL, int NV, int P, bool WIDE>
__device__ __forceinline__ void vec_dots(const VecRows<WEL> &w, const VecToken<WEL, WIDE> (*x)[P], int n,
                                         float (*acc)[NV * P]) {
#pragma unroll
  for (int r = 0; r < kVecRows; ++r) {
    if constexpr (WIDE && WEL == EL_F16) {
#pragma unroll
      for (int c = 0; c < NV; ++c)
        if (c < n)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const f16x8_t h = __builtin_bit_cast(f16x8_t, w.r[r]);
            acc[r][c] = fmaf((float)h[i], __int_as_float(x[c][0].v[i >> 2][i & 3]), acc[r][c]);
          }
    } else if constexpr (is_mx(WEL)) {
      const float f = __uint_as_float((uint32_t)w.s[r] << 23);
      int q[8];  // 16 codes as bf16 pairs, exact there
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = w.r[r][i];
        q[2 * i] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, f, false));
        q[2 * i + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, f, true));
      }
#pragma unroll
      for (int c = 0; c < NV; ++c)
        if (c < n)
#pragma unroll
          for (int d = 0; d < P; ++d)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              acc[r][c * P + d] = dot2<EL>(q[i], x[c][d].v[i >> 2][i & 3], acc[r][c * P + d]);
      __builtin_amdgcn_sched_barrier(0);  // one row's expanded codes in registers at a time
    } else {
#pragma unroll
      for (int c = 0; c < NV; ++c)
        if (c < n)
#pragma unroll
          for (int d = 0; d < P; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int a = w.r[r][i], b = x[c][d].v[0][i];
              float &s = acc[r][c * P + d];
              if constexpr (EL == EL_F32) s = fmaf(__int_as_float(a), __int_as_float(b), s);
              else s = dot2<EL>(a, b, s);
            }
    }
  }
}

// Sums over the wave's lanes of 8 values: lane l gets that of value vec_row(l).  Each of
// the first steps adds two values' halves of the lanes, so the values halve with it.
__device__ __forceinline__ int vec_row(int lane) { return (lane >> 5) * 4 + ((lane >> 4) & 1) * 2 + ((lane >> 3) & 1); }
template <int dpp>
__device__ __forceinline__ float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), dpp, 0xf, 0xf, true));
}
__device__ __forceinline__ float vec_sum(const float *v, int stride) {
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i * stride]), __float_as_uint(v[(i + 4) * stride]),
                                                    false, false);
    a[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[i]), __float_as_uint(a[i + 2]), false, false);
    b[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  const bool high = threadIdx.x & 8;
  float s = (high ? b[1] : b[0]) + dpp_move<0x128>(high ? b[0] : b[1]);  // rotate by 8 within 16
  s += dpp_move<0xb1>(s);   // quad_perm [1, 0, 3, 2]
  s += dpp_move<0x4e>(s);   // quad_perm [2, 3, 0, 1]
  s += dpp_move<0x141>(s);  // mirrored within 8: the other quad
  return s;
}

// Token's value a for slot's row of the workspace, column f.
template <int EL>
__device__ __forceinline__ void store_a(const MoeParams &p, int slot, int64_t f, float a) {
  const int64_t at = slot * p.F + f;
  if constexpr (EL != EL_BF16) {
    ((float *)p.a)[at] = a;
  } else {
    uint16_t *hi = (uint16_t *)p.a, *lo = hi + (int64_t)p.T * p.k * p.F;
    split(a, hi[at], lo[at]);
  }
}

// Bytes of a row of a (bf16: of one of its planes).
template <int EL>
__device__ __forceinline__ uint32_t a_row_bytes(int64_t F) { return (uint32_t)(F * (EL == EL_BF16 ? 2 : 4)); }

__device__ __forceinline__ float swiglu(float g, float u) { return g * sigmoid(g) * u; }

// The 8 rows of W1 behind 4 columns of a, a wave's share of the workgroup's.
template <int WEL>
struct UpRows {
  __amdgpu_buffer_rsrc_t wg, wu, sg, su;
  int64_t f0;
  uint32_t wb;
  int n;  // columns below F
  __device__ UpRows(const MoeParams &p, int e, int64_t f) : f0(f), wb((uint32_t)row_bytes<WEL>(p.K)) {
    n = (int)(p.F - f < 4 ? p.F - f : 4);
    wg = moe_rsrc(weight_row<WEL>(p.w1, e, f));
    wu = moe_rsrc(weight_row<WEL>(p.w1, e, p.F + f));
    sg = moe_rsrc(is_mx(WEL) ? scale_row(p.w1, e, f) : nullptr);
    su = moe_rsrc(is_mx(WEL) ? scale_row(p.w1, e, p.F + f) : nullptr);
  }
  __device__ void load(VecRows<WEL> &w, int block) const {
    const uint32_t at = (block * 64 + (threadIdx.x & 63)) * 16;
    w.load(wg, sg, 0, 4, at, wb, n);
    w.load(wu, su, 4, 4, at, wb, n);
  }
};

// a of 4 columns f0 ... f0 + 3 for up to NV tokens, by one wave: rows 0-3 are the gate's,
// 4-7 the up's.
template <int EL, int WEL, int NV>
__device__ __forceinline__ void up_vector(const MoeParams &p, const UpTokens &tok, const UpRows<WEL> &rows,
                                          VecRows<WEL> &w0) {
  const int lane = threadIdx.x & 63;
  constexpr uint32_t kX = 16 * VecToken<WEL>::parts;
  const uint32_t xb = (uint32_t)(p.K * elem_bytes(EL));
  const auto xr = moe_rsrc(p.x);
  uint32_t xrow[NV];
#pragma unroll
  for (int c = 0; c < NV; ++c) xrow[c] = __builtin_amdgcn_readfirstlane(tok.slot[c < tok.n ? c : 0] / p.k) * xb;
  float acc[kVecRows][NV] = {};
  const int blocks = (int)((p.K + block_elems<WEL>() - 1) / block_elems<WEL>());
  VecToken<WEL> x0[NV][1], x1[NV][1];
  const auto load_x = [&](VecToken<WEL> (*x)[1], int b) {
#pragma unroll
    for (int c = 0; c < NV; ++c)
      if (c < tok.n) x[c][0].load(xr, xrow[c], (b * 64 + lane) * kX, xb);
  };
  VecRows<WEL> w1;
  load_x(x0, 0);
  for (int b = 0; b < blocks; b += 2) {  // two register sets in turn
    load_x(x1, b + 1);
    rows.load(w1, b + 1);
    __builtin_amdgcn_sched_barrier(0);
    vec_dots<EL, WEL, NV>(w0, x0, tok.n, acc);
    if (b + 1 >= blocks) break;
    __builtin_amdgcn_sched_barrier(0);
    load_x(x0, b + 2);
    rows.load(w0, b + 2);
    __builtin_amdgcn_sched_barrier(0);
    vec_dots<EL, WEL, NV>(w1, x1, tok.n, acc);
    __builtin_amdgcn_sched_barrier(0);
  }
  const int64_t f = rows.f0 + (vec_row(lane) & 3);
  const bool mine = lane < 32 && f < p.F;
  const float bg = mine ? bias_at<EL>(p.w1, tok.expert, f) : 0.f, bu = mine ? bias_at<EL>(p.w1, tok.expert, p.F + f) : 0.f;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    if (c >= tok.n) break;
    const float g = vec_sum(&acc[0][c], NV), u = __shfl_xor(g, 32);
    if (mine && (lane & 7) == 0) store_a<EL>(p, tok.slot[c], f, tok.gate[c] * swiglu(g + bg, u + bu));
  }
}

// ----------------------------------------------------------------- many columns --
// Contraction over K for up to NT tiles of 16 columns (HIGH false: one of 8): wave w takes
// units (MXFP8: pairs of units) w, w + kUpWaves, ... of the gate's and the up's 16 rows, U of
// each at a time.
template <int EL, int WEL, int NT, bool HIGH>
__device__ __forceinline__ void up_product(const MoeParams &p, const UpTokens &tok, int64_t f0, float *sums) {
  using W = Unit<WEL, kMoeRows>;
  constexpr int U = up_units<WEL>();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = tok.expert;
  const WeightLane rows(p.F - f0, (uint32_t)row_bytes<WEL>(p.K), p.K);
  const auto wg = moe_rsrc(weight_row<WEL>(p.w1, e, f0)), wu = moe_rsrc(weight_row<WEL>(p.w1, e, p.F + f0));
  const auto sg = moe_rsrc(is_mx(WEL) ? scale_row(p.w1, e, f0) : nullptr);
  const auto su = moe_rsrc(is_mx(WEL) ? scale_row(p.w1, e, p.F + f0) : nullptr);
  // units past the end load zeros; scales: the unit is the first of a pair
  const auto load = [&](W *g, W *u, int c0, auto scales) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t at = (uint32_t)(c0 + i * kUpWaves) * 128;
      g[i].load(wg, sg, rows, at);
      u[i].load(wu, su, rows, at);
    }
    if constexpr (W::pairs && scales()) {
      g->load_scales(sg, rows, (uint32_t)c0 * 128);
      u->load_scales(su, rows, (uint32_t)c0 * 128);
    }
  };
  static_assert(!W::pairs || U == 1, "a pair is two steps");
  W g[U], u[U], ng[U], nu[U];
  load(g, u, W::pairs ? 2 * wave : wave, std::true_type());
  const uint32_t xb = (uint32_t)(p.K * elem_bytes(EL));
  const auto xr = moe_rsrc(p.x);
  uint32_t xrow[NT][2], xend[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = t * 16 + h * 8 + (lane & 7);
      xend[t][h] = c < tok.n ? xb : 0;
      xrow[t][h] = c < tok.n ? (uint32_t)(tok.slot[c] / p.k) * xb : 0;
    }
  f32x4_t ag[NT], au[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) ag[t] = au[t] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  const int units = (int)((p.K + W::kElems - 1) / W::kElems);
  const auto step = [&](int c0, int next, W *g, W *u, W *ng, W *nu, auto first) {
    uint32_t at[U];
#pragma unroll
    for (int i = 0; i < U; ++i) at[i] = (uint32_t)(c0 + i * kUpWaves) * W::b_bytes;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t && t * 16 >= tok.n) break;
      // the tokens' pieces come from cache, the next weights from memory: issued in this
      // order, the products wait for the former alone
      Columns<W, U, HIGH> b;
      b.load(xr, xrow[t][0], xend[t][0], xrow[t][1], xend[t][1], at);
      if (t == 0) load(ng, nu, next, std::bool_constant<!first()>());
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (W::pairs && first())
        if (t == 0) {
          g->take_scales(rows, (uint32_t)c0 * 128, *ng);
          u->take_scales(rows, (uint32_t)c0 * 128, *nu);
        }
#pragma unroll
      for (int i = 0; i < U * W::steps; ++i) {
        const i32x4_t x = b.operand(i);
        ag[t] = mma<EL>(g[i / W::steps].operand(i % W::steps), x, ag[t]);
        au[t] = mma<EL>(u[i / W::steps].operand(i % W::steps), x, au[t]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // two register sets in turn: copying one to the other would wait for its loads
  constexpr int kNext = W::pairs ? 1 : kUpWaves * U;
  for (int c0 = W::pairs ? 2 * wave : wave; c0 < units; c0 += 2 * kUpWaves * U) {
    step(c0, c0 + kNext, g, u, ng, nu, std::true_type());
    if (c0 + kNext >= units) break;
    step(c0 + kNext, c0 + 2 * kUpWaves * U, ng, nu, g, u, std::false_type());
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float *o = sums + (((t * kUpWaves + wave) * 2) * 64 + lane) * 4;
    *(f32x4_t *)o = ag[t];
    *(f32x4_t *)(o + 256) = au[t];
  }
}

// a of the workgroup's 16 columns for all of the expert's tokens.
template <int EL, int WEL, int NT>
__device__ __forceinline__ void up_many(const MoeParams &p, const UpTokens &tok, int64_t f0, float *sums) {
  if (tok.n <= 8) up_product<EL, WEL, 1, false>(p, tok, f0, sums);
  else up_product<EL, WEL, NT, true>(p, tok, f0, sums);
  __syncthreads();
  const int f = threadIdx.x & 15;
  if (f0 + f >= p.F) return;
  const float bg = bias_at<EL>(p.w1, tok.expert, f0 + f), bu = bias_at<EL>(p.w1, tok.expert, p.F + f0 + f);
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
    store_a<EL>(p, tok.slot[c], f0 + f, tok.gate[c] * swiglu(g, u));
  }
}

// Without MFMA the waves share nothing but the search, and smaller workgroups spread more
// evenly (one token, 8 experts of 2048/768, 768 workgroups of two waves: 11.8 us, 384 of four
// 13.2).
template <int NT>
constexpr int up_threads() { return NT ? kUpThreads : kUpThreads / 2; }
// Waves a SIMD that the registers have to allow: three (17 tokens over 32 experts of 4096/2048
// in MXFP8 codes: 74 us, 81 at the two that the compiler settles for), for which two tiles of
// MXFP8 codes spill 8 registers; four tiles would spill more.
template <int NT>
constexpr int up_waves() { return NT == 1 || NT == 2 ? 3 : 1; }

// NV: experts of up to that many tokens go by up_vector, the others by up_product in at
// most NT tiles (NT 0: the call has no more than NV tokens).
template <int EL, int WEL, int NV, int NT>
__global__ __launch_bounds__(up_threads<NT>(), up_waves<NT>()) void moe_up_kernel(const MoeParams p) {
  __shared__ UpTokens tok;
  __shared__ __align__(16) float sums[NT ? NT * kUpWaves * 2 * 64 * 4 : 4];
  const int lane = threadIdx.x & 63;
  const int64_t f0 = (int64_t)blockIdx.x * (up_threads<NT>() / 16);
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
  const UpRows<WEL> rows(p, valid ? e : 0, f0 + (threadIdx.x >> 6) * 4);
  VecRows<WEL> r;
  // a slot's expert is almost always read: its first rows are on their way during the
  // search for its tokens
  if (NV > 0 && valid && !by_expert) rows.load(r, 0);
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
  if constexpr (NV > 0) {
    if (NT == 0 || tok.n <= NV) {
      if (by_expert) rows.load(r, 0);
      up_vector<EL, WEL, NV>(p, tok, rows, r);
      return;
    }
  }
  if constexpr (NT > 0) up_many<EL, WEL, NT>(p, tok, f0, sums);
}

// LDS of the down kernel: the entries with an expert, in order.
struct DownEntry {
  int32_t expert;
  int32_t base, n;  // its tokens' slots are slots[base ... base + n)
};

// A workgroup's place in the down kernel: its first row of W2, and its tables in LDS.
struct DownPlace {
  int64_t n0;
  const DownEntry *ent;  // n_vec entries of few tokens from the front, the others from the back
  const int16_t *slots;
  float *acc;  // [waves][T][16 rows] sums of a token
  int n_vec, n_many;
};

// Entries of up to NV tokens: items (entry, 8 rows, 1 KiB block of F), dealt to the waves
// in turn.
template <int EL, int WEL, int R, int NV>
__device__ __forceinline__ void down_vector(const MoeParams &p, const DownPlace &o) {
  constexpr int parts = EL == EL_BF16 ? 2 : 1;  // of a
  using Token = VecToken<WEL, is_mx(WEL) || EL == EL_F16>;
  constexpr uint32_t kX = 16 * Token::parts;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t wb = (uint32_t)row_bytes<WEL>(p.F), ab = a_row_bytes<EL>(p.F);
  const uint32_t plane = (uint32_t)(p.T * p.k) * ab;
  const auto ar = moe_rsrc(p.a);
  const int blocks = (int)((p.F + block_elems<WEL>() - 1) / block_elems<WEL>()), per = blocks * (R / 8);
  int i = wave / per, c = wave - i * per;
  const auto load = [&](VecRows<WEL> &w, Token (*x)[parts], int i, int c) {
    const int h = c / blocks, b = c - h * blocks;
    const DownEntry t = o.ent[i];
    const int e = __builtin_amdgcn_readfirstlane(t.expert), n = __builtin_amdgcn_readfirstlane(t.n);
    const int base = __builtin_amdgcn_readfirstlane(t.base);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (k < n) {
        const uint32_t row = (uint32_t)__builtin_amdgcn_readfirstlane(o.slots[base + k]) * ab;
#pragma unroll
        for (int d = 0; d < parts; ++d) x[k][d].load(ar, row + d * plane, (b * 64 + lane) * kX, ab);
      }
    const int64_t r0 = o.n0 + h * 8;
    w.load(moe_rsrc(weight_row<WEL>(p.w2, e, r0)), moe_rsrc(is_mx(WEL) ? scale_row(p.w2, e, r0) : nullptr), 0, 8,
           (uint32_t)(b * 64 + lane) * 16, wb, (int)min64(p.N - r0, 8));
  };
  const auto step = [&](const VecRows<WEL> &w, const Token (*x)[parts], VecRows<WEL> &nw, Token (*nx)[parts]) {
    int ni = i, nc = c + kDownWaves;
    while (nc >= per) {
      nc -= per;
      ++ni;
    }
    if (ni < o.n_vec) load(nw, nx, ni, nc);
    __builtin_amdgcn_sched_barrier(0);
    const int n = __builtin_amdgcn_readfirstlane(o.ent[i].n), base = __builtin_amdgcn_readfirstlane(o.ent[i].base);
    float acc[kVecRows][NV * parts] = {};
    vec_dots<EL, WEL, NV>(w, x, n, acc);
    if constexpr (parts == 2)
#pragma unroll
      for (int r = 0; r < kVecRows; ++r)
#pragma unroll
        for (int j = 0; j < NV; ++j) acc[r][j * parts] = join(acc[r][j * parts], acc[r][j * parts + 1]);
    // lanes 0 ... 7 of a row's 8 hold the same sum: the k-th adds token k's
    const int k = lane & 7;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j < n) {
        const float v = vec_sum(&acc[0][j * parts], NV * parts);
        sum = k == j ? v : sum;
      }
    if (k < n) o.acc[(wave * p.T + o.slots[base + k] / p.k) * 16 + (c / blocks) * 8 + vec_row(lane)] += sum;
    __builtin_amdgcn_sched_barrier(0);
    i = ni;
    c = nc;
  };
  VecRows<WEL> w0, w1;
  Token x0[NV][parts], x1[NV][parts];
  if (i < o.n_vec) load(w0, x0, i, c);
  while (i < o.n_vec) {  // two register sets in turn
    step(w0, x0, w1, x1);
    if (i >= o.n_vec) break;
    step(w1, x1, w0, x0);
  }
}

// The other entries: items (entry, U units of F), dealt to the waves in turn, 16 rows by
// the entry's tokens in MFMA steps.  The branches around the next item's loads (the last item,
// an array of addresses, the loop over tokens) make the compiler wait for them before the
// products, so a CU's other waves cover a step's time.  Without them (loads that go nowhere
// after the last item, addresses by scalar loads, the first tokens apart) small layers gained
// and large ones lost: 20 tokens over 32 experts of 2048/1024 in fp32 184 -> 172 us, 64 over
// 256 of 7168/2048 in bf16 3.02 -> 3.12 ms, 64 over 8 of 4096/14336 in fp16 703 -> 716 us.
template <int EL, int WEL, int R>
__device__ __forceinline__ void down_many(const MoeParams &p, const DownPlace &o) {
  using W = Unit<WEL, R>;
  constexpr int U = kDownUnits;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const auto entry = [&](int i) { return o.ent[p.n_entries - 1 - i]; };
  const uint32_t ab = a_row_bytes<EL>(p.F);
  const WeightLane rows(min64(p.N - o.n0, R), (uint32_t)row_bytes<WEL>(p.F), p.F);
  const auto ar = moe_rsrc(p.a);
  constexpr int kCols = EL == EL_F32 ? 16 : 8;  // tokens of a step
  const uint32_t plane = (uint32_t)(p.T * p.k) * ab;  // from a's first parts to the second
  const int pieces = (int)((p.F + W::kElems * U - 1) / (W::kElems * U));
  const auto load = [&](W *w, int i, int c) {
    const int e = __builtin_amdgcn_readfirstlane(entry(i).expert);
    const auto r = moe_rsrc(weight_row<WEL>(p.w2, e, o.n0));
    const auto s = moe_rsrc(is_mx(WEL) ? scale_row(p.w2, e, o.n0) : nullptr);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      w[j].load(r, s, rows, (c * U + j) * 128);
      if constexpr (W::pairs)
        if (j % 2 == 0) w[j].load_scales(s, rows, (c * U + j) * 128);
    }
  };
  int i = wave / pieces, c = wave - i * pieces;
  // one item with its weights in `cur`; moves on to the next, whose weights go to `nxt`
  const auto step = [&](W *cur, W *nxt) {
    int ni = i, nc = c + kDownWaves;
    while (nc >= pieces) {
      nc -= pieces;
      ++ni;
    }
    const int base = __builtin_amdgcn_readfirstlane(entry(i).base), m = __builtin_amdgcn_readfirstlane(entry(i).n);
    uint32_t at[U];
#pragma unroll
    for (int j = 0; j < U; ++j) at[j] = (c * U + j) * W::b_bytes;
    // the entry's tokens as columns; for 16-bit products a's two parts are columns of a step
    for (int t = 0; t < m; t += kCols) {
      const int lo = t + (lane & 7), hi = kCols == 16 ? lo + 8 : lo;
      const uint32_t row_lo = lo < m ? (uint32_t)o.slots[base + lo] * ab : 0;
      const uint32_t row_hi = kCols == 8 ? row_lo + plane : hi < m ? (uint32_t)o.slots[base + hi] * ab : 0;
      std::conditional_t<EL == EL_F16, ScaledColumns<W, U>, Columns<W, U, true>> b;
      if constexpr (EL == EL_F16) b.load(ar, row_lo, lo < m ? ab : 0, at);
      else b.load(ar, row_lo, lo < m ? ab : 0, row_hi, hi < m ? ab : 0, at);
      if (t == 0 && ni < o.n_many) load(nxt, ni, nc);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (W::pairs)
        if (t == 0)
#pragma unroll
          for (int j = 0; j < U; j += 2) cur[j].take_scales(rows, (c * U + j) * 128, cur[j + 1]);
      if constexpr (EL == EL_F16) b.split();
      f32x4_t sum = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < U * W::steps; ++s) sum = mma<EL>(cur[s / W::steps].operand(s % W::steps), b.operand(s), sum);
      if constexpr (kCols == 8)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float rest = __shfl_xor(sum[r], 8);
          if constexpr (EL == EL_F16) sum[r] = b.sum(sum[r], rest);
          else sum[r] = join(sum[r], rest);
        }
      if (col < kCols && t + col < m) {  // each column another token: no lane shares a sum
        f32x4_t *to = (f32x4_t *)(o.acc + (wave * p.T + o.slots[base + t + col] / p.k) * 16 + q * 4);
        *to += sum;
      }
    }
    i = ni;
    c = nc;
  };
  // two register sets in turn: copying one to the other would wait for its loads
  W w0[U], w1[U];
  if (i < o.n_many) load(w0, i, c);
  while (i < o.n_many) {
    step(w0, w1);
    if (i >= o.n_many) break;
    step(w1, w0);
  }
}

template <int EL, int WEL, int R, int NV, bool MANY>
__global__ __launch_bounds__(kDownThreads) void moe_down_kernel(const MoeParams p) {
  extern __shared__ __align__(16) char lds[];
  __shared__ int3 wave_n[kDownWaves];
  float *acc = (float *)lds;  // [waves][T][16 rows] sums of a token
  DownEntry *ent = (DownEntry *)(acc + kDownWaves * p.T * 16);
  int16_t *slots = (int16_t *)(ent + p.n_entries);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * R;
  for (int i = threadIdx.x; i < kDownWaves * p.T * 4; i += kDownThreads) ((f32x4_t *)acc)[i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  // compact the table: running counts of the entries of few tokens, the others, and of all
  // their tokens
  int n_vec = 0, n_many = 0, members = 0;
  for (int d0 = 0; d0 < p.n_entries; d0 += kDownThreads) {
    const int d = d0 + threadIdx.x;
    MoeEntry t{0, -1, 0};
    if (d < p.n_entries) t = p.entries[d];
    const int mine = t.expert >= 0 ? __popcll(t.tokens) : 0;
    const bool few = mine > 0 && (!MANY || mine <= NV);
    const uint64_t vec = __ballot(few), many = __ballot(mine > 0 && !few), below = (1ull << lane) - 1;
    int upto = mine;  // inclusive sum over the wave's lanes
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(upto, s);
      if (lane >= s) upto += o;
    }
    if (lane == 63) wave_n[wave] = make_int3(__popcll(vec), __popcll(many), upto);
    __syncthreads();
    int at_vec = n_vec + __popcll(vec & below), at_many = n_many + __popcll(many & below);
    int base = members + upto - mine;
    for (int w = 0; w < kDownWaves; ++w) {
      const int3 n = wave_n[w];
      if (w < wave) {
        at_vec += n.x;
        at_many += n.y;
        base += n.z;
      }
      n_vec += n.x;
      n_many += n.y;
      members += n.z;
    }
    if (mine) {
      ent[few ? at_vec : p.n_entries - 1 - at_many] = {t.expert, base, mine};
      slots[base] = (int16_t)t.first;
      uint64_t left = t.tokens & (t.tokens - 1);
      for (int i = base + 1; left; ++i, left &= left - 1)
        slots[i] = p.slot_of[d * 64 + __ffsll((unsigned long long)left) - 1];
    }
    __syncthreads();
  }
  const DownPlace place{n0, ent, slots, acc, n_vec, n_many};
  if constexpr (NV > 0) down_vector<EL, WEL, R, NV>(p, place);
  if constexpr (MANY) down_many<EL, WEL, R>(p, place);
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
  const auto go_up = [&](auto nv, auto nt) {
    constexpr int threads = up_threads<nt()>(), columns = threads / 16;
    hipLaunchKernelGGL((moe_up_kernel<EL, WEL, nv(), nt()>), dim3((unsigned)((p.F + columns - 1) / columns), p.n_entries),
                       dim3(threads), 0, s, p);
  };
  using std::integral_constant;
  using Zero = integral_constant<int, 0>;
  using One = integral_constant<int, 1>;
  using Two = integral_constant<int, 2>;
  using Four = integral_constant<int, 4>;
  // Dot products where the whole call has as few tokens: up to four of 16-bit or fp32 weights
  // in the up kernel (4 tokens over 8 experts of 4096/8192: 127 us, by MFMA 136), two
  // otherwise (down kernel, 2 tokens there: 63 us, by MFMA 85).  In larger calls only beside
  // MXFP8 codes, for the experts of one or two tokens, where the MFMA's columns would load
  // 256 bytes of activations for every 128 of codes (8 tokens over 32 experts of 4096/1920:
  // up 53.5 us, all by MFMA 55.7; 17 over 32 of 4096/2048: down 44.3 and 46.1; bf16 does as
  // well by MFMA), and in the down kernel beside fp16 weights, whose MFMA steps have to split a
  // (calls of 5 tokens over 8 experts of 4096/14336: 374 us, all by MFMA 384; 32 tokens, top 6
  // of 64 experts of 2048/1408: 227 and 249; 64 over the 8: 703 both).
  using Few = integral_constant<int, is_mx(WEL) ? 2 : 0>;
  using FewDown = integral_constant<int, is_mx(WEL) || EL == EL_F16 ? 2 : 0>;
  if (p.T == 1) go_up(One(), Zero());
  else if (p.T == 2) go_up(Two(), Zero());
  else if (p.T <= 4 && !is_mx(WEL)) go_up(integral_constant<int, is_mx(WEL) ? 2 : 4>(), Zero());
  else if (p.T <= 16) go_up(Few(), One());
  else if (p.T <= 32) go_up(Few(), Two());
  else go_up(Few(), Four());

  // LDS: at most 4 KiB of sums a wave, 24 KiB of entries and 4 KiB of slots
  const size_t lds = (size_t)kDownWaves * p.T * 64 + (size_t)p.n_entries * sizeof(DownEntry) + (size_t)p.T * p.k * 2;
  const auto go_down = [&](auto r, auto nv, auto many) {
    hipLaunchKernelGGL((moe_down_kernel<EL, WEL, r(), nv(), many()>), dim3((unsigned)((p.N + r() - 1) / r())),
                       dim3(kDownThreads), lds, s, p);
  };
  // Rows of a workgroup: 8 as long as no CU gets a second one (call over 64 experts of 2048/768,
  // top 8: 16 tokens into N = 2048 117 us, by 16 rows 125; into 1024 109 and 121), else 16, whose
  // loads share the tokens' between more rows (64 tokens over 32 experts of 2880/2880 into 2880:
  // 367 us, by 8 rows 456; 17 tokens in MXFP8 codes, 32 experts of 4096/2048, into 2176: 150 and
  // 167).  The short workgroups of one token go without MXFP8 codes as well by two on a CU (one
  // token, 64 experts of 2048/768, into 4032: 8 rows 25.0 us, 16 26.3; into 7168 33.7 and 31.6).
  const auto by_tokens = [&](auto r) {
    if (p.T == 1) go_down(r, One(), std::false_type());
    else if (p.T == 2) go_down(r, Two(), std::false_type());
    else go_down(r, FewDown(), std::true_type());
  };
  if (p.N <= 8 * kCUs || (p.T == 1 && !is_mx(WEL) && p.N < 16 * kCUs)) by_tokens(integral_constant<int, 8>());
  else by_tokens(integral_constant<int, 16>());
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
  if (mx && K % 128 == 0 && F % 128 == 0 && K > 128 && F > 128) launch_moe_typed<EL_BF16, EL_MX>(p, s);
  else if (mx) launch_moe_typed<EL_BF16, EL_MX_RAGGED>(p, s);
  else if (el == EL_F32) launch_moe_typed<EL_F32, EL_F32>(p, s);
  else if (el == EL_F16) launch_moe_typed<EL_F16, EL_F16>(p, s);
  else launch_moe_typed<EL_BF16, EL_BF16>(p, s);
  return hipGetLastError();
}

}  // namespace gl
