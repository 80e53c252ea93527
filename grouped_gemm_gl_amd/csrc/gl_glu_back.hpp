// The two products of the gated layer's backward on small tiles: dx = dh W_g (rows grouped) and
// dW_g = dh^T x (the contraction grouped), for fp32 and for problems whose 256-row tiles would be too
// few to fill the chip.
//
// Both are out[i][j] = sum_p A(i, p) B(p, j) with j contiguous in B and out; A is dh, contiguous in
// p for dx and in i for dW.  Tiles of TI x TJ outputs: 64 x 64 (4 waves, two workgroups a CU), dx also
// 32 x 64 (4 waves, three; or with the contraction in two parts 8, one), or 128 x 128 (8 waves);
// stages of the contraction (64 values of 16 bits, 32 of 32) go straight to a ring of STAGES in LDS,
// STAGES - 1 ahead, one barrier a stage (as in glu_mid_kernel).  An operand whose tile index is
// contiguous is staged as it lies, contraction row after contraction row, and turned on the way out of LDS: 16-bit values by the transposing read, which hands a lane 4 contraction values
// of one column, 32-bit ones by single-word reads.  16-byte slots are permuted by the row so that
// the rows a read touches lie in different banks.
//
// Rows past the contraction's end are outside the stage's buffer resource and load zeros, columns
// past the matrix take an offset outside.  Sums are fp32 in a fixed order (deterministic).
#pragma once

#include "gl_glu_tile.hpp"

namespace gl {

// ONCE: dx's weights are loaded as data that is read once, fp32 weight gradients stored as data that is
// not read soon.
// PARTS of dx's contraction, as in glu_mid_kernel.
template <int IN, int EL, bool WGRAD, int TI, int TJ, int STAGES, bool ONCE, int PARTS>
__global__ __launch_bounds__((PARTS * MidTile<TI, TJ>::kThreads), 2) void glu_back_kernel(BackParams p) {
  using Op = Operand<IN>;
  using M = MidTile<TI, TJ, STAGES>;
  using Tn = Turned<IN, TJ>;  // dW: of A too, TI is TJ
  static_assert(!WGRAD || TI == TJ, "square tiles");
  constexpr int E = in_bytes(IN);
  constexpr int kRing = M::kStages * M::kStageBytes;
  __shared__ __attribute__((aligned(1024))) char lds[PARTS * kRing];

  const WsView ws = ws_view(p.ws, p.G);
  const RowTiles tiles(ws, p.G, TI);
  if (!ws_usable(ws.hdr, p.G, p.T)) return;
  const int tiles_i = (int)((p.N + TI - 1) / TI), tiles_j = (int)((p.K + TJ - 1) / TJ);
  const int64_t total = WGRAD ? (int64_t)p.G * tiles_i * tiles_j : (int64_t)tiles.tile(p.G) * tiles_j;
  const int lane = threadIdx.x & 63;
  const int index = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = PARTS == 1 ? 0 : index / M::kWaves, wave = PARTS == 1 ? index : index % M::kWaves;
  char *const ring = lds + part * kRing;
  const int wm = wave & 1, wn = wave >> 1;
  const int fr = lane & 15, fq = lane >> 4;
  const int64_t kbytes = p.K * E, nbytes = p.N * E;

  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    int g, it, jt;
    if (WGRAD) {
      const int per = tiles_i * tiles_j;
      g = (int)(w / per);
      const int l = (int)(w - (int64_t)g * per);
      it = l / tiles_j;
      jt = l - it * tiles_j;
    } else {
      const int qt = (int)(w / tiles_j);
      jt = (int)(w - (int64_t)qt * tiles_j);
      g = tiles.group(qt);
      if (!device_check(g >= 0 && g < p.G, p.ws)) continue;
      it = qt - tiles.tile(g);
    }
    const int64_t g_off = tiles.row(g), g_rows = tiles.row(g + 1) - g_off;
    if (WGRAD && p.accumulate && g_rows == 0) continue;  // not touched
    const int64_t i0 = (int64_t)it * TI, j0 = (int64_t)jt * TJ;
    const int64_t contr = WGRAD ? g_rows : p.N;  // values of the contraction
    const int rows = (int)min64(TI, (WGRAD ? p.N : g_rows) - i0), cols = (int)min64(TJ, p.K - j0);
    if (!device_check(rows > 0 && cols > 0 && g_off >= 0 && g_rows >= 0 && g_off + g_rows <= p.T, p.ws)) continue;
    const char *a = WGRAD ? p.a + g_off * nbytes + i0 * E : p.a + (g_off + i0) * nbytes;
    const char *b = WGRAD ? p.x + g_off * kbytes
                          : p.b ? p.b + (int64_t)g * p.N * kbytes : p.b_ptrs[g];
    b += j0 * E;
    const int stages = (int)((contr + Tn::kRows - 1) / Tn::kRows), nk = (stages + PARTS - 1) / PARTS;  // nk of each part
    const int64_t part0 = (int64_t)part * nk * Tn::kRows;

    // K-major A: pieces of 8 rows, 128 bytes of each; turned operands: pieces of kPieceRows rows
    const int c16 = ((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7)) * 16;
    auto issue = [&](int s) {
      char *st = ring + (s % M::kStages) * M::kStageBytes;
      const int64_t first = part0 + (int64_t)s * Tn::kRows;
      const int left = s < nk && (PARTS == 1 || first < contr) ? (int)min64(Tn::kRows, contr - first) : 0;  // contraction values of the stage
      auto turned = [&](const char *base, int64_t ld, int width, char *to) {
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            (void *)gemm::uniform_ptr(base + (left > 0 ? first * ld : 0)), (short)0, (int)(max(left, 1) * ld), 0x00020000);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int u = wave + q * M::kWaves, row = u * Tn::kPieceRows + lane / Tn::kSlots;
          const int c = Tn::slot(row, lane % Tn::kSlots) * 16;  // its own inverse
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              r, (GL_LDS void *)(to + u * 1024), 16,
              row < left && c < width * E ? (uint32_t)(row * (int)ld + c) : kPastEnd, 0, 0, ONCE && !WGRAD ? 2 : 0);
        }
      };
      if constexpr (WGRAD) {
        turned(a, nbytes, rows, st);
      } else {
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void *)gemm::uniform_ptr(a), (short)0,
                                                                           (int)(rows * nbytes), 0x00020000);
#pragma unroll
        for (int q = 0; q < M::kRowPieces; ++q) {
          const int u = wave + q * M::kWaves;
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              r, (GL_LDS void *)(st + u * 1024), 16,
              c16 < left * E ? (uint32_t)((8 * u + (lane >> 3)) * (int)nbytes + c16) : kPastEnd,
              left > 0 ? (int)(first * E) : 0, 0, 0);
        }
      }
      turned(b, kbytes, cols, st + TI * 128);
    };
    const int blocks = (rows - wm * 16 + 31) / 32;
    f32x4_t acc[2][M::kBlocks];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < M::kBlocks; ++i) acc[h][i] = f32x4_t{0, 0, 0, 0};
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
      // read_turned waits for its reads, so what is multiplied next is read before
      i32x4_t fb[2][2], fa[M::kBlocks][2];
      if constexpr (IN != IN_F32) {
        const uint32_t at[2] = {Tn::address(st + TI * 128, wn * 32, lane), Tn::address(st + TI * 128, wn * 32 + 16, lane)};
        if constexpr (WGRAD) {
          uint32_t ata[M::kBlocks];
#pragma unroll
          for (int i = 0; i < M::kBlocks; ++i) ata[i] = Tn::address(st, i * 32 + wm * 16, lane);
          read_turned<Tn::kRow>(ata, fa);
        }
        read_turned<Tn::kRow>(at, fb);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 2; ++c) fb[h][c] = Tn::frag(st + TI * 128, wn * 32 + h * 16, c, lane);
      }
#pragma unroll
      for (int i = 0; i < M::kBlocks; ++i) {
        if (i >= blocks) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if constexpr (!WGRAD) {
            const int r = i * 32 + wm * 16 + fr;
            fa[i][c] = *(const i32x4_t *)(st + r * 128 + (((4 * c + fq) ^ ((r >> 1) & 7)) << 4));
          } else if constexpr (IN == IN_F32) {
            fa[i][c] = Tn::frag(st, i * 32 + wm * 16, c, lane);
          }
          acc[0][i] = Op::mma(fb[0][c], fa[i][c], acc[0][i]);
          acc[1][i] = Op::mma(fb[1][c], fa[i][c], acc[1][i]);
        }
      }
      sums.step(s, kFp32Chain / 32, &acc[0][0]);
    }
    sums.end(&acc[0][0]);
    if constexpr (PARTS == 2) add_parts<2 * M::kBlocks>(lds, part, wave, lane, &acc[0][0]);
    void *out = WGRAD && !p.out ? p.out_ptrs[g] : p.out;
    const int64_t out0 = WGRAD ? (p.out ? (int64_t)g * p.N * p.K : 0) + i0 * p.K : (g_off + i0) * p.K;
#pragma unroll
    for (int i = 0; i < M::kBlocks; ++i) {
      const int rl = i * 32 + wm * 16 + fr;
      if (rl >= rows || part != 0) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = wn * 32 + h * 16 + fq * 4;
        if (c >= cols) continue;
        const int64_t at = out0 + rl * p.K + j0 + c;
        float4 v = make_float4(acc[h][i][0], acc[h][i][1], acc[h][i][2], acc[h][i][3]);
        if (WGRAD && p.accumulate) {
          const float4 o = load4<EL>(out, at);
          v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
        }
        if constexpr (WGRAD && ONCE) {
          static_assert(EL == EL_F32, "fp32 gradients");
          __builtin_nontemporal_store(f32x4_t{v.x, v.y, v.z, v.w}, (f32x4_t *)((float *)out + at));
        } else {
          put4<EL>(out, at, v);
        }
      }
    }
    gemm::wait_vm0();
    __syncthreads();
  }
}

template <int IN, int EL, bool WGRAD, int TI, int TJ = TI, int STAGES = 4, bool ONCE = false, int PARTS = 1>
inline hipError_t launch_glu_back_tile(const BackParams &p, hipStream_t s) {
  const int64_t tiles_j = (p.K + TJ - 1) / TJ, groups = p.T < p.G ? p.T : p.G;
  const int64_t items = WGRAD ? p.G * ((p.N + TI - 1) / TI) * tiles_j : ((p.T + TI - 1) / TI + groups) * tiles_j;
  hipLaunchKernelGGL((glu_back_kernel<IN, EL, WGRAD, TI, TJ, STAGES, ONCE, PARTS>), dim3((unsigned)(items < 8192 ? items : 8192)),
                     dim3(PARTS * MidTile<TI, TJ>::kThreads), 0, s, p);
  return hipGetLastError();
}

// The instances of choose_glu_back (gl_glu_choice.hpp).
template <int IN, int EL>
inline hipError_t launch_glu_back(const BackParams &p, bool wgrad, bool out_f32, hipStream_t s) {
  const BackChoice c = choose_glu_back(IN, wgrad, out_f32, p.G, p.T, p.K, p.N);
  if constexpr (IN == IN_F32) {
    if (wgrad)
      return c.once ? launch_glu_back_tile<IN, EL, true, 64, 64, 3, true>(p, s)
                    : launch_glu_back_tile<IN, EL, true, 64, 64, 3>(p, s);
    if (c.parts == 2) return launch_glu_back_tile<IN, EL, false, 32, 64, 4, false, 2>(p, s);
    if (c.rows == 32)
      return c.once ? launch_glu_back_tile<IN, EL, false, 32, 64, 4, true>(p, s)
                    : launch_glu_back_tile<IN, EL, false, 32, 64>(p, s);
    return c.once ? launch_glu_back_tile<IN, EL, false, 64, 64, 4, true>(p, s)
                  : launch_glu_back_tile<IN, EL, false, 64>(p, s);
  } else {
    GluParams q{};
    q.x = p.a; q.ws = p.ws; q.G = p.G; q.T = p.T; q.F = p.K; q.out = p.out; q.out_ptrs = p.out_ptrs;
    if (!wgrad) {
      if (c.rows == 256) {
        q.w = p.b; q.w_ptrs = p.b_ptrs; q.K = p.N;
        return launch_glu_tile<IN, EL, EPI_DX, ACT_SILU>(q, c.items, c.tiles, s);
      }
      if (c.rows == 128)
        return c.once ? launch_glu_back_tile<IN, EL, false, 128, 128, 4, true>(p, s)
                      : launch_glu_back_tile<IN, EL, false, 128>(p, s);
      return c.rows == 32 ? launch_glu_back_tile<IN, EL, false, 32, 64, 4, false, 2>(p, s)
                          : launch_glu_back_tile<IN, EL, false, 64>(p, s);
    }
    if (c.rows == 256) {
      q.w = p.x; q.N = p.N; q.accumulate = p.accumulate;
      return out_f32 ? launch_glu_tile<IN, EL_F32, EPI_DW, ACT_SILU>(q, c.items, c.tiles, s)
                     : launch_glu_tile<IN, EL, EPI_DW, ACT_SILU>(q, c.items, c.tiles, s);
    }
    if (c.rows == 128)
      return out_f32 ? launch_glu_back_tile<IN, EL_F32, true, 128>(p, s) : launch_glu_back_tile<IN, EL, true, 128>(p, s);
    return out_f32 ? launch_glu_back_tile<IN, EL_F32, true, 64>(p, s) : launch_glu_back_tile<IN, EL, true, 64>(p, s);
  }
}

}  // namespace gl
