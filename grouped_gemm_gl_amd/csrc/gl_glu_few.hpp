// The fp32 gated products for at most 16 rows in all and few columns: one row tile a group, and not
// enough of it to fill the chip, so the contraction is split too.
//
// A workgroup of four waves takes 16 columns of the gate and the 16 of the other half that
// belong to them of one group.  Its waves split the contraction: wave v takes
// units v, v + 4, .., a unit being 128 bytes of every row, straight from memory to registers as
// whole 128-byte lines (8 rows a load, and a rotation of 8 lanes gives the matrix instruction its
// layout).  The weights are the instruction's first operand and the rows its second, so a lane
// ends with four neighbouring columns of a row.  The four waves' sums meet in LDS and are added in
// a fixed order.
//
// Bound by the latency of a few loads one after the other: 8 rows on 4 groups, K 1024 F 512, 9.1 us a call,
// 13.6 on tiles of 32 by 64 with the contraction in two parts.  (16 bits and 8-bit integers, whose stages
// hold two and four times the values, go by those tiles: 6.3 us both, 2 groups of 16, K 2048 F 2048 bf16 8.9
// here and 7.9 there, but one of 16, K 4096 F 4096 14.8 and 15.4.)
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

template <int EPI>
__global__ __launch_bounds__(kFewThreads) void glu_few_kernel(GluParams p) {
  constexpr int IN = IN_F32, EL = EL_F32, kCols = 16;
  using Op = Operand<IN>;
  using acc_t = typename Op::acc_t;
  __shared__ acc_t part[kFewWaves][2][64];
  const WsView ws = ws_view(p.ws, p.G);
  const RowTiles tiles(ws, p.G, 32);
  if (!ws_usable(ws.hdr, p.G, p.T)) return;
  const int tiles_j = (int)((p.F + kCols - 1) / kCols);
  const int64_t total = (int64_t)tiles.tile(p.G) * tiles_j;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const uint32_t kb = (uint32_t)(p.K * in_bytes(IN));  // bytes of a row of either operand
  const uint32_t chunk = (r >> 3) * 64 + q * 16;       // the lane's place in a unit

  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int qt = (int)(w / tiles_j), jt = (int)(w - (int64_t)qt * tiles_j);
    const int g = tiles.group(qt);
    if (!device_check(g >= 0 && g < p.G, p.ws)) continue;
    const int64_t row0 = tiles.row(g);
    const int rows = (int)min64(16, tiles.row(g + 1) - row0);
    if (!device_check(rows > 0 && row0 >= 0 && row0 + rows <= p.T && qt == tiles.tile(g), p.ws)) continue;
    const int64_t col0 = (int64_t)jt * kCols;
    const char *wg = group_weights<IN, EPI>(p, g);
    const int64_t second = p.F + col0;
    const int cols = (int)min64(16, p.F - col0);
    const __amdgpu_buffer_rsrc_t w0 = few_rsrc(wg + col0 * kb);
    const __amdgpu_buffer_rsrc_t w1 = few_rsrc(wg + second * kb);
    const uint32_t low = (r & 7) * kb + chunk, high = low + 8 * kb;
    const bool loww = (r & 7) < cols, highw = (r & 7) + 8 < cols;

    const __amdgpu_buffer_rsrc_t xr = few_rsrc(p.x + row0 * kb);
    const bool lowx = (r & 7) < rows, highx = (r & 7) + 8 < rows;
    acc_t acc[2] = {acc_t{0, 0, 0, 0}, acc_t{0, 0, 0, 0}};
    struct Unit {
      RowBlock g, u, x;
    };
    auto load = [&](Unit &n, uint32_t at) {
      const bool in = at + chunk < kb;
      n.g.load(w0, in && loww ? low + at : kPastEnd, in && highw ? high + at : kPastEnd);
      n.u.load(w1, in && loww ? low + at : kPastEnd, in && highw ? high + at : kPastEnd);
      n.x.load(xr, in && lowx ? low + at : kPastEnd, in && highx ? high + at : kPastEnd);
    };
    auto multiply = [&](const Unit &n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const i32x4_t xv = n.x.chunk(c);
        acc[0] = Op::mma(n.g.chunk(c), xv, acc[0]);
        acc[1] = Op::mma(n.u.chunk(c), xv, acc[1]);
      }
    };
    // two units in turn, so the next one's loads are in flight during a unit's products; a
    // unit past the row's end loads zeros
    constexpr uint32_t step = kFewWaves * 128;
    Unit u0, u1;
    uint32_t at = wave * 128;
    load(u0, at);
    load(u1, at + step);
    ChunkSums<IN, 2> sums;
    for (int n = 0; at < kb; at += 2 * step, ++n) {
      multiply(u0);
      load(u0, at + 2 * step);
      multiply(u1);
      load(u1, at + 3 * step);
      sums.step(n, kFp32Chain / 64, acc);
    }
    sums.end(acc);
    part[wave][0][lane] = acc[0];
    part[wave][1][lane] = acc[1];
    __syncthreads();
    if (wave == 0 && r < rows) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int v = 1; v < kFewWaves; ++v) acc[h] += part[v][h][lane];
      const int64_t row = row0 + r;
      const int c = 4 * q;
      if (c < cols) {
        const float4 v0 = finish<IN, EL>(acc[0], RowScale(), column_terms<IN, EL, EPI>(p, g, col0 + c));
        const float4 v1 = finish<IN, EL>(acc[1], RowScale(), column_terms<IN, EL, EPI>(p, g, second + c));
        with_activation(p.act, [&](auto act) { gated4<EL, EPI, decltype(act)::value>(p, row, col0 + c, v0, v1); });
      }
    }
    __syncthreads();
  }
}

template <int EPI>
inline hipError_t launch_glu_few(const GluParams &p, hipStream_t s) {
  const int64_t items = (p.T < p.G ? p.T : p.G) * ((p.F + 15) / 16);
  hipLaunchKernelGGL((glu_few_kernel<EPI>), dim3((unsigned)(items < 4096 ? items : 4096)), dim3(kFewThreads), 0,
                     s, p);
  return hipGetLastError();
}

}  // namespace gl
