// Grouped products with a gated or scaled epilogue on small tiles, where 256-row tiles would be
// too few to fill the chip: 32 rows by 32 weight rows (2 waves, five workgroups a CU) or by 64 (4
// waves, three), either also with the contraction in two parts (twice the waves and LDS), 64 by 64
// (4 waves, two) or 128 by 128 (8 waves, one); half of the weight rows the gate's and half the
// other's of the same columns (plain: neighbouring columns).
//
// Stages of 128 bytes of every row go straight to a ring of kStages in LDS, kStages - 1 ahead, and
// one barrier a stage does for both sides: after it every wave's loads of the stage are there,
// and every wave has read the stage before, whose place the next loads take.  Waves are 2 by
// WAVES / 2; a wave has every other block of 16 rows (those past the tile's last row are skipped)
// by 16 columns of either half, so h_g and h_u are in the same lane.
//
// Bound by the weights' bytes in flight: 64 groups, 4099 rows, K 2048 F 1400, fp16, 172 us for 734 MB
// (4.3 TB/s from HBM, tiles of 128); 32 of 64 rows, K 1408 N 2048, int8, 13.6 us for 73 MB (5.4 TB/s, most of it
// from the last-level cache, 32 by 64).  A ring of five stages was slower, of three (fp32, three workgroups a CU) 5%
// slower at 333 rows and up to 7% faster at more.
#pragma once

#include "gl_gemm_tile.hpp"
#include "gl_glu_few.hpp"

namespace gl {

// 64 (or 32) contraction rows of TILE columns in LDS, as they lie in memory.
template <int IN, int TILE>
struct Turned {
  static constexpr int E = in_bytes(IN), kRow = TILE * E, kRows = 128 / E;
  static constexpr int kPieceRows = 1024 / kRow, kSlots = kRow / 16;
  // slot of the 16-byte chunk c of row p.  16-bit: a read's half wave touches 2 chunks of the rows
  // 4 t + 0..3 and 8 + 4 t + 0..3; 32-bit: 4 chunks of four rows that are 4 apart.
  __device__ static __forceinline__ int slot(int p, int c) {
    if (IN == IN_F32) return c ^ (((p >> 2) & 3) << 2);
    if (kRow == 128) return c ^ ((((p >> 1) & 1) | (((p >> 3) & 1) << 1)) << 1);
    return c ^ (((p & 3) | (((p >> 3) & 1) << 2)) << 1);
  }
  // 32-bit: 16 bytes of column col + l % 16, contraction values 4 (l / 16) .. + 3 of the stage's half c
  // (of 16)
  __device__ static __forceinline__ i32x4_t frag(const char *st, int col, int c, int lane) {
    const int q = lane & 15, g = lane >> 4;
    i32x4_t o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = 16 * c + 4 * g + e, at = (col + q) * 4;
      o[e] = *(const int *)(st + p * kRow + (slot(p, at >> 4) << 4) + (at & 15));
    }
    return o;
  }
  // 16-bit: the lane's place in the stage for the transposing reads of columns col .. + 15.  Lane q of a group of
  // 16 names row q / 4 and columns 4 (q % 4) .. + 3 of four rows, and gets column q of them; group g
  // takes the rows 8 g .. + 7 of a half of 32 in two reads.
  __device__ static __forceinline__ uint32_t place(int col, int lane) {
    const int q = lane & 15, g = lane >> 4, p = 8 * g + (q >> 2), at = (col + ((q & 3) << 2)) * 2;
    return p * kRow + (slot(p, at >> 4) << 4) + (at & 15);
  }
  __device__ static __forceinline__ uint32_t address(const char *st, int col, int lane) {
    return (uint32_t)(uintptr_t)(GL_LDS const char *)st + place(col, lane);
  }
};

// The fragments of B blocks of 16 columns, both halves of a stage: contraction values 8 (l / 16) ..
// + 7 of column l % 16.  In one asm block with its wait: before the builtin the compiler waits for all
// loads to LDS that are under way, the next stages' too.
template <int ROW, int B>
__device__ __forceinline__ void read_turned(const uint32_t (&at)[B], i32x4_t (&o)[B][2]) {
  typedef __attribute__((ext_vector_type(2))) int i32x2_t;
  i32x2_t v[B][4];
#define GL_TR(n) "ds_read_b64_tr_b16 %" #n ", "
  if constexpr (B == 2) {
    asm volatile(GL_TR(0) "%8\n\t" GL_TR(1) "%8 offset:%c10\n\t" GL_TR(2) "%8 offset:%c11\n\t" GL_TR(3) "%8 offset:%c12\n\t"
                 GL_TR(4) "%9\n\t" GL_TR(5) "%9 offset:%c10\n\t" GL_TR(6) "%9 offset:%c11\n\t" GL_TR(7) "%9 offset:%c12\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[0][2]), "=&v"(v[0][3]), "=&v"(v[1][0]), "=&v"(v[1][1]),
                   "=&v"(v[1][2]), "=&v"(v[1][3])
                 : "v"(at[0]), "v"(at[1]), "n"(4 * ROW), "n"(32 * ROW), "n"(36 * ROW)
                 : "memory");
  } else {
    static_assert(B == 4, "blocks");
    asm volatile(GL_TR(0) "%16\n\t" GL_TR(1) "%16 offset:%c20\n\t" GL_TR(2) "%16 offset:%c21\n\t" GL_TR(3) "%16 offset:%c22\n\t"
                 GL_TR(4) "%17\n\t" GL_TR(5) "%17 offset:%c20\n\t" GL_TR(6) "%17 offset:%c21\n\t" GL_TR(7) "%17 offset:%c22\n\t"
                 GL_TR(8) "%18\n\t" GL_TR(9) "%18 offset:%c20\n\t" GL_TR(10) "%18 offset:%c21\n\t" GL_TR(11) "%18 offset:%c22\n\t"
                 GL_TR(12) "%19\n\t" GL_TR(13) "%19 offset:%c20\n\t" GL_TR(14) "%19 offset:%c21\n\t" GL_TR(15) "%19 offset:%c22\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[0][2]), "=&v"(v[0][3]), "=&v"(v[1][0]), "=&v"(v[1][1]),
                   "=&v"(v[1][2]), "=&v"(v[1][3]), "=&v"(v[2][0]), "=&v"(v[2][1]), "=&v"(v[2][2]), "=&v"(v[2][3]),
                   "=&v"(v[3][0]), "=&v"(v[3][1]), "=&v"(v[3][2]), "=&v"(v[3][3])
                 : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(4 * ROW), "n"(32 * ROW), "n"(36 * ROW)
                 : "memory");
  }
#undef GL_TR
#pragma unroll
  for (int b = 0; b < B; ++b)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      o[b][c] = i32x4_t{v[b][2 * c][0], v[b][2 * c][1], v[b][2 * c + 1][0], v[b][2 * c + 1][1]};
}

template <int ROWS, int WEIGHT_ROWS = ROWS, int STAGES = 4>
struct MidTile {
  static constexpr int kWaves = WEIGHT_ROWS / 16, kThreads = 64 * kWaves;
  static constexpr int kStages = STAGES;
  static constexpr int kStageBytes = (ROWS + WEIGHT_ROWS) * 128;  // rows, then weight rows
  static constexpr int kRowPieces = ROWS / 8 / kWaves, kPieces = kRowPieces + 2;  // of 1 KiB, of a wave
  static constexpr int kBlocks = ROWS / 32;  // of 16 rows, of a wave
  static constexpr int kColsHalf = WEIGHT_ROWS / 2;  // weight rows of a half
  static_assert(kPieces * kWaves * 1024 == kStageBytes && kColsHalf == 16 * (kWaves / 2), "waves cover the tile");
};

// The contraction in two parts: twice the waves, the second half of which goes through the second half
// of the stages in a ring of its own; its sums are added to the first's, in LDS, in a fixed order.
// add_parts is called by every wave, after which those of part 0 have the sums.
template <int N, class acc_t>
__device__ __forceinline__ void add_parts(char *lds, int part, int wave, int lane, acc_t *acc) {
  gemm::wait_vm0();
  __syncthreads();  // the ring is not in use any more
  acc_t *sums = (acc_t *)lds + wave * N * 64 + lane;
  if (part == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) sums[i * 64] = acc[i];
  }
  __syncthreads();
  if (part == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += sums[i * 64];
  }
}

// ONCE: the weights are loaded as data that is read once; PARTS of the contraction (see choose_glu).
template <int IN, int EL, int EPI, int ROWS, int WEIGHT_ROWS, bool ONCE, int PARTS>
__global__ __launch_bounds__((PARTS * MidTile<ROWS, WEIGHT_ROWS>::kThreads), 2) void glu_mid_kernel(GluParams p) {
  using Op = Operand<IN>;
  using acc_t = typename Op::acc_t;
  using M = MidTile<ROWS, WEIGHT_ROWS>;
  constexpr int kCols = EPI == EPI_PLAIN ? 2 * M::kColsHalf : M::kColsHalf;
  constexpr int kRing = M::kStages * M::kStageBytes;
  __shared__ __attribute__((aligned(1024))) char lds[PARTS * kRing];

  const WsView ws = ws_view(p.ws, p.G);
  const RowTiles tiles(ws, p.G, ROWS);
  if (!ws_usable(ws.hdr, p.G, p.T)) return;
  const int tiles_j = (int)((p.F + kCols - 1) / kCols);
  const int64_t total = (int64_t)tiles.tile(p.G) * tiles_j;
  const int lane = threadIdx.x & 63;
  const int index = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = PARTS == 1 ? 0 : index / M::kWaves, wave = PARTS == 1 ? index : index % M::kWaves;
  const int wm = wave & 1, wn = wave >> 1;
  const int fr = lane & 15, fq = lane >> 4;
  const int kb = (int)(p.K * in_bytes(IN));
  const int stages = (kb + 127) / 128, nk = (stages + PARTS - 1) / PARTS, part0 = part * nk * 128;  // nk of each part
  char *const ring = lds + part * kRing;
  // pieces of 8 rows: wave w has the pieces w and (not in 32 rows by 64) w + kWaves of the rows, and
  // piece w of each half of the weight rows
  const int c16 = ((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7)) * 16;
  const uint32_t voff = (uint32_t)(8 * wave + (lane >> 3)) * (uint32_t)kb + (uint32_t)c16;

  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int qt = (int)(w / tiles_j), jt = (int)(w - (int64_t)qt * tiles_j);
    const int g = tiles.group(qt);
    if (!device_check(g >= 0 && g < p.G, p.ws)) continue;
    const int64_t row0 = tiles.row(g) + (int64_t)(qt - tiles.tile(g)) * ROWS;
    const int rows = (int)min64(ROWS, tiles.row(g + 1) - row0);
    if (!device_check(rows > 0 && row0 >= 0 && row0 + rows <= p.T, p.ws)) continue;
    const int64_t col0 = (int64_t)jt * kCols, left = p.F - col0;
    const int64_t second = EPI == EPI_PLAIN ? col0 + M::kColsHalf : p.F + col0;
    const char *wg = group_weights<IN, EPI>(p, g);
    auto rsrc = [&](const char *at, int64_t n) {
      return __builtin_amdgcn_make_buffer_rsrc((void *)gemm::uniform_ptr(at), (short)0, (int)n * kb, 0x00020000);
    };
    const bool has1 = EPI != EPI_PLAIN || left > M::kColsHalf;
    const __amdgpu_buffer_rsrc_t rx = rsrc(p.x + row0 * kb, rows);
    const __amdgpu_buffer_rsrc_t r0 = rsrc(wg + col0 * kb, min64(M::kColsHalf, left));
    // (no second half: one row of the first, whose products are not stored)
    const __amdgpu_buffer_rsrc_t r1 =
        has1 ? rsrc(wg + second * kb, min64(M::kColsHalf, EPI == EPI_PLAIN ? left - M::kColsHalf : left))
             : rsrc(wg + col0 * kb, 1);
    auto issue = [&](int s) {
      char *st = ring + (s % M::kStages) * M::kStageBytes;
      const int at = part0 + s * 128, lim = s < nk ? kb - at : 0;
      const uint32_t far = (uint32_t)(8 * M::kWaves) * (uint32_t)kb;  // from a wave's piece of a half to its next
      const uint32_t o0 = c16 < lim ? voff : kPastEnd, o1 = c16 < lim ? voff + far : kPastEnd;
      const int soff = lim > 0 ? at : 0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (GL_LDS void *)(st + wave * 1024), 16, o0, soff, 0, 0);
      if constexpr (M::kRowPieces == 2)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (GL_LDS void *)(st + (wave + M::kWaves) * 1024), 16, o1, soff, 0, 0);
      char *wt = st + ROWS * 128 + wave * 1024;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r0, (GL_LDS void *)wt, 16, o0, soff, 0, ONCE ? 2 : 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r1, (GL_LDS void *)(wt + M::kWaves * 1024), 16, o0, soff, 0, ONCE ? 2 : 0);
    };
    const int blocks = (rows - wm * 16 + 31) / 32;  // of the wave that hold rows
    acc_t acc[2][M::kBlocks];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < M::kBlocks; ++i) acc[h][i] = acc_t{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < M::kStages - 1; ++s) issue(s);
    ChunkSums<IN, 2 * M::kBlocks> sums;
    for (int s = 0; s < nk; ++s) {
      __builtin_amdgcn_sched_barrier(0);
      gemm::wait_vm<(M::kStages - 2) * M::kPieces>();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      issue(s + M::kStages - 1);
      const char *st = ring + (s % M::kStages) * M::kStageBytes;
      auto frag = [&](int row, int c) {
        const int r = row + fr;
        return *(const i32x4_t *)(st + r * 128 + (((4 * c + fq) ^ ((r >> 1) & 7)) << 4));
      };
      i32x4_t b[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) b[h][c] = frag(ROWS + h * M::kColsHalf + wn * 16, c);
#pragma unroll
      for (int i = 0; i < M::kBlocks; ++i) {
        if (i >= blocks) break;
        const i32x4_t a0 = frag(i * 32 + wm * 16, 0), a1 = frag(i * 32 + wm * 16, 1);
        acc[0][i] = Op::mma(b[0][0], a0, acc[0][i]);
        acc[1][i] = Op::mma(b[1][0], a0, acc[1][i]);
        acc[0][i] = Op::mma(b[0][1], a1, acc[0][i]);
        acc[1][i] = Op::mma(b[1][1], a1, acc[1][i]);
      }
      sums.step(s, kFp32Chain / 32, &acc[0][0]);
    }
    sums.end(&acc[0][0]);
    if constexpr (PARTS == 2) add_parts<2 * M::kBlocks>(lds, part, wave, lane, &acc[0][0]);
    const int c = wn * 16 + fq * 4;
    const bool in0 = c < left && part == 0, in1 = EPI == EPI_PLAIN ? c + M::kColsHalf < left : in0;
    if (in0) {
      const ColumnTerms<IN, EL> t0 = column_terms<IN, EL, EPI>(p, g, col0 + c);
      const ColumnTerms<IN, EL> t1 = column_terms<IN, EL, EPI>(p, g, in1 ? second + c : col0 + c);
      auto finish_all = [&](auto act) {
#pragma unroll
        for (int i = 0; i < M::kBlocks; ++i) {
          const int rl = i * 32 + wm * 16 + fr;
          if (rl >= rows) break;
          const int64_t row = row0 + rl;
          const RowScale rs(IN == IN_I8 ? p.x_scale[row] : 0.f);
          const float4 v0 = finish<IN, EL>(acc[0][i], rs, t0), v1 = finish<IN, EL>(acc[1][i], rs, t1);
          if constexpr (EPI == EPI_PLAIN) {
            put4<EL>(p.out, row * p.F + col0 + c, v0);
            if (in1) put4<EL>(p.out, row * p.F + second + c, v1);
          } else {
            gated4<EL, EPI, decltype(act)::value>(p, row, col0 + c, v0, v1);
          }
        }
      };
      if constexpr (EPI == EPI_PLAIN) finish_all(std::integral_constant<int, ACT_SILU>{});
      else with_activation(p.act, finish_all);
    }
    // the loads past the last stage (zeros) are done, and every wave has read, before the ring is
    // filled again or the workgroup ends
    gemm::wait_vm0();
    __syncthreads();
  }
}

template <int IN, int EL, int EPI, int ROWS, int WEIGHT_ROWS, int PARTS = 1>
inline hipError_t launch_glu_mid(const GluParams &p, bool once, hipStream_t s) {
  using M = MidTile<ROWS, WEIGHT_ROWS>;
  constexpr int kCols = EPI == EPI_PLAIN ? 2 * M::kColsHalf : M::kColsHalf;
  const int64_t groups = p.T < p.G ? p.T : p.G;
  const int64_t items = ((p.T + ROWS - 1) / ROWS + groups) * ((p.F + kCols - 1) / kCols);
  const dim3 grid((unsigned)(items < 8192 ? items : 8192)), block(PARTS * M::kThreads);
  if constexpr (PARTS == 1) {  // (in two parts the weights are few)
    if (once) {
      hipLaunchKernelGGL((glu_mid_kernel<IN, EL, EPI, ROWS, WEIGHT_ROWS, true, PARTS>), grid, block, 0, s, p);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((glu_mid_kernel<IN, EL, EPI, ROWS, WEIGHT_ROWS, false, PARTS>), grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace gl
