// Grouped products with a gated or scaled epilogue for few rows a group (decoding): bound by
// reading the used groups' weights once.
//
// A workgroup of four waves takes 16 columns of the gate and the 16 of the other half that
// belong to them (plain: 32 columns), for up to 16 NB rows of one group.  Its waves split the
// contraction: wave v takes units v, v + 4, .., a unit being 128 bytes of every row, straight
// from memory to registers as whole 128-byte lines (8 rows a load, and a rotation of 8 lanes
// gives the matrix instruction its layout).  The weights are the instruction's first operand
// and the rows its second, so a lane ends with four neighbouring columns of a row.  The four
// waves' sums meet in LDS and are added in a fixed order.
#pragma once

#include "gl_glu.hpp"

namespace gl {

constexpr int kFewWaves = 4, kFewThreads = 64 * kFewWaves;
constexpr uint32_t kPastEnd = 0x80000000u;  // an offset past every resource: the load gives zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t few_rsrc(const void *base) {
  const uint64_t v = (uint64_t)(uintptr_t)base;  // the same in every lane; made visibly so
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void *)(uintptr_t)(((uint64_t)hi << 32) | lo), (short)0, 0x7fffffff,
                                           0x00020000);
}

// 16 rows x 128 bytes of an operand: `low` holds rows 0-7, `high` rows 8-15, lanes r and r + 8
// sharing a row; chunk(h) is the lane's 16 bytes of row l % 16, of the unit's half h.
struct RowBlock {
  i32x4_t low, high;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at_low, uint32_t at_high) {
    low = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)at_low, 0, 0));
    high = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)at_high, 0, 0));
  }
  __device__ __forceinline__ i32x4_t chunk(int h) const {
    i32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // row_ror:8 into the lanes of rows 8-15, or 0-7
      o[i] = h == 0 ? __builtin_amdgcn_update_dpp(low[i], high[i], 0x128, 0xf, 0xc, false)
                    : __builtin_amdgcn_update_dpp(high[i], low[i], 0x128, 0xf, 0x3, false);
    return o;
  }
};

// NB: blocks of 16 rows that an item takes at most; 16 NB <= tile_rows, the height of the row
// tiles that the items are counted in.
template <int IN, int EL, int EPI, int NB>
__global__ __launch_bounds__(kFewThreads) void glu_few_kernel(GluParams p, int tile_rows) {
  using Op = Operand<IN>;
  using acc_t = typename Op::acc_t;
  constexpr int kCols = EPI == EPI_PLAIN ? 32 : 16;
  __shared__ acc_t part[kFewWaves][2][NB][64];
  const WsView ws = ws_view(p.ws, p.G);
  if (!ws_usable(ws.hdr, p.G, p.T)) return;
  const int64_t *__restrict__ off = ws.off;
  const int32_t *__restrict__ pre = ws.pre[tile_rows_index(tile_rows)];
  const int tiles_j = (int)((p.F + kCols - 1) / kCols);
  const int64_t total = (int64_t)pre[p.G] * tiles_j;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const uint32_t kb = (uint32_t)(p.K * in_bytes(IN));  // bytes of a row of either operand
  const uint32_t chunk = (r >> 3) * 64 + q * 16;       // the lane's place in a unit

  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int qt = (int)(w / tiles_j), jt = (int)(w - (int64_t)qt * tiles_j);
    const int g = find_group(pre, p.G, qt);
    if (!device_check(g >= 0 && g < p.G, p.ws)) continue;
    const int64_t g_off = off[g], in_group = (int64_t)(qt - pre[g]) * tile_rows;
    const int64_t rows = min64(tile_rows, off[g + 1] - g_off - in_group), row0 = g_off + in_group;
    if (!device_check(rows > 0 && row0 >= 0 && row0 + rows <= p.T, p.ws)) continue;
    const int64_t col0 = (int64_t)jt * kCols;
    // weight rows of the first 16 columns and of the second: the other half, or the next 16
    const char *wg = group_weights<IN, EPI>(p, g);
    const int64_t second = EPI == EPI_PLAIN ? col0 + 16 : p.F + col0;
    const int cols0 = (int)min64(16, p.F - col0);
    const int cols1 = EPI == EPI_PLAIN ? (int)max((int64_t)0, min64(16, p.F - second)) : cols0;
    const __amdgpu_buffer_rsrc_t w0 = few_rsrc(wg + col0 * kb);
    const __amdgpu_buffer_rsrc_t w1 = few_rsrc(wg + (cols1 > 0 ? second : col0) * kb);
    const uint32_t low = (r & 7) * kb + chunk, high = low + 8 * kb;
    const bool low0 = (r & 7) < cols0, high0 = (r & 7) + 8 < cols0;
    const bool low1 = (r & 7) < cols1, high1 = (r & 7) + 8 < cols1;

    for (int64_t first = 0; first < rows; first += 16 * NB) {
      const __amdgpu_buffer_rsrc_t xr = few_rsrc(p.x + (row0 + first) * kb);
      const int left = (int)min64(16 * NB, rows - first);
      acc_t acc[2][NB];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[h][b] = acc_t{0, 0, 0, 0};
      struct Unit {
        RowBlock g, u, x[NB];
      };
      auto load = [&](Unit &n, uint32_t at) {
        const bool in = at + chunk < kb;
        n.g.load(w0, in && low0 ? low + at : kPastEnd, in && high0 ? high + at : kPastEnd);
        n.u.load(w1, in && low1 ? low + at : kPastEnd, in && high1 ? high + at : kPastEnd);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int xl = b * 16 + (r & 7);
          n.x[b].load(xr, in && xl < left ? (uint32_t)xl * kb + chunk + at : kPastEnd,
                      in && xl + 8 < left ? (uint32_t)(xl + 8) * kb + chunk + at : kPastEnd);
        }
      };
      auto multiply = [&](const Unit &n) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const i32x4_t wg_ = n.g.chunk(c), wu_ = n.u.chunk(c);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const i32x4_t xv = n.x[b].chunk(c);
            acc[0][b] = Op::mma(wg_, xv, acc[0][b]);
            acc[1][b] = Op::mma(wu_, xv, acc[1][b]);
          }
        }
      };
      // two units in turn, so the next one's loads are in flight during a unit's products; a
      // unit past the row's end loads zeros
      constexpr uint32_t step = kFewWaves * 128;
      Unit u0, u1;
      uint32_t at = wave * 128;
      load(u0, at);
      load(u1, at + step);
      for (; at < kb; at += 2 * step) {
        multiply(u0);
        load(u0, at + 2 * step);
        multiply(u1);
        load(u1, at + 3 * step);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) part[wave][h][b][lane] = acc[h][b];
      __syncthreads();
      for (int b = wave; b < NB; b += kFewWaves) {
        acc_t s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s[h] = part[0][h][b][lane];
#pragma unroll
          for (int v = 1; v < kFewWaves; ++v) s[h] += part[v][h][b][lane];
        }
        const int xl = b * 16 + r;
        if (xl >= left) continue;
        const int64_t row = row0 + first + xl;
        const float rs = IN == IN_I8 ? p.x_scale[row] : 0.f;
        const int c = 4 * q;
        if constexpr (EPI == EPI_PLAIN) {
          if (c < cols0)
            put4<EL>(p.out, row * p.F + col0 + c, finish<IN, EL>(s[0], rs, column_terms<IN, EL, EPI>(p, g, col0 + c)));
          if (c < cols1)
            put4<EL>(p.out, row * p.F + second + c, finish<IN, EL>(s[1], rs, column_terms<IN, EL, EPI>(p, g, second + c)));
        } else if (c < cols0) {
          const float4 v0 = finish<IN, EL>(s[0], rs, column_terms<IN, EL, EPI>(p, g, col0 + c));
          const float4 v1 = finish<IN, EL>(s[1], rs, column_terms<IN, EL, EPI>(p, g, second + c));
          with_activation(p.act, [&](auto act) { gated4<EL, EPI, decltype(act)::value>(p, row, col0 + c, v0, v1); });
        }
      }
      __syncthreads();
    }
  }
}

template <int IN, int EL, int EPI>
inline hipError_t launch_glu_few(const GluParams &p, hipStream_t s) {
  constexpr int kCols = EPI == EPI_PLAIN ? 32 : 16;
  const int64_t groups = p.T < p.G ? p.T : p.G;
  auto grid = [&](int tile) {
    const int64_t items = ((p.T + tile - 1) / tile + groups) * ((p.F + kCols - 1) / kCols);
    return dim3((unsigned)(items < 4096 ? items : 4096));
  };
  if (p.T <= 16)
    hipLaunchKernelGGL((glu_few_kernel<IN, EL, EPI, 1>), grid(32), dim3(kFewThreads), 0, s, p, 32);
  else
    hipLaunchKernelGGL((glu_few_kernel<IN, EL, EPI, 4>), grid(64), dim3(kFewThreads), 0, s, p, 64);
  return hipGetLastError();
}

}  // namespace gl
