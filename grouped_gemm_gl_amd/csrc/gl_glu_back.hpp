// The two products of the gated layer's backward on small tiles: dx = dh W_g (rows grouped) and
// dW_g = dh^T x (the contraction grouped), for fp32 and for problems whose 256-row tiles would be too
// few to fill the chip.
//
// Both are out[i][j] = sum_p A(i, p) B(p, j) with j contiguous in B and out; A is dh, contiguous in
// p for dx and in i for dW.  Tiles of TILE x TILE outputs, TILE 64 (4 waves, two workgroups a CU)
// or 128 (8 waves); stages of the contraction (64 values of 16 bits, 32 of 32) go straight to a
// ring of four in LDS, three ahead, one barrier a stage (as in glu_mid_kernel).  An operand whose tile
// index is contiguous is staged as it lies, contraction row after contraction row, and turned on
// the way out of LDS: 16-bit values by the transposing read, which hands a lane 4 contraction values
// of one column, 32-bit ones by single-word reads.  16-byte slots are permuted by the row so that
// the rows a read touches lie in different banks.
//
// Rows past the contraction's end are outside the stage's buffer resource and load zeros, columns
// past the matrix take an offset outside.  Sums are fp32 in a fixed order (deterministic).
#pragma once

#include "gl_glu_mid.hpp"

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
  // 16 bytes of column col + l % 16: 16-bit, contraction values 8 (l / 16) .. + 7 of the stage's half c
  // (of 32); 32-bit, 4 (l / 16) .. + 3 of the half (of 16)
  __device__ static __forceinline__ i32x4_t frag(const char *st, int col, int c, int lane) {
    const int q = lane & 15, g = lane >> 4;
    i32x4_t o;
    if constexpr (IN == IN_F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = 16 * c + 4 * g + e, at = (col + q) * 4;
        o[e] = *(const int *)(st + p * kRow + (slot(p, at >> 4) << 4) + (at & 15));
      }
    } else {
      const int at = (col + ((q & 3) << 2)) * 2;
      gemm::v4i16 h[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int p = 32 * c + 8 * g + 4 * t + (q >> 2);
        h[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (GL_LDS gemm::v4i16 *)(st + p * kRow + (slot(p, at >> 4) << 4) + (at & 15)));
      }
      const gemm::v8i16 v = {h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
      o = __builtin_bit_cast(i32x4_t, v);
    }
    return o;
  }
};

template <int IN, int EL, bool WGRAD, int TILE>
__global__ __launch_bounds__(MidTile<TILE>::kThreads, 2) void glu_back_kernel(BackParams p) {
  using Op = Operand<IN>;
  using M = MidTile<TILE>;
  using Tn = Turned<IN, TILE>;
  constexpr int E = in_bytes(IN);
  __shared__ __attribute__((aligned(1024))) char lds[M::kStages * M::kStageBytes];

  const WsView ws = ws_view(p.ws, p.G);
  if (!ws_usable(ws.hdr, p.G, p.T)) return;
  const int64_t *__restrict__ off = ws.off;
  const int32_t *__restrict__ pre = ws.pre[tile_rows_index(TILE)];
  const int tiles_i = (int)((p.N + TILE - 1) / TILE), tiles_j = (int)((p.K + TILE - 1) / TILE);
  const int64_t total = WGRAD ? (int64_t)p.G * tiles_i * tiles_j : (int64_t)pre[p.G] * tiles_j;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
      g = find_group(pre, p.G, qt);
      if (!device_check(g >= 0 && g < p.G, p.ws)) continue;
      it = qt - pre[g];
    }
    const int64_t g_off = off[g], g_rows = off[g + 1] - g_off;
    if (WGRAD && p.accumulate && g_rows == 0) continue;  // not touched
    const int64_t i0 = (int64_t)it * TILE, j0 = (int64_t)jt * TILE;
    const int64_t contr = WGRAD ? g_rows : p.N;  // values of the contraction
    const int rows = (int)min64(TILE, (WGRAD ? p.N : g_rows) - i0), cols = (int)min64(TILE, p.K - j0);
    if (!device_check(rows > 0 && cols > 0 && g_off >= 0 && g_off + g_rows <= p.T, p.ws)) continue;
    const char *a = WGRAD ? p.a + g_off * nbytes + i0 * E : p.a + (g_off + i0) * nbytes;
    const char *b = WGRAD ? p.x + g_off * kbytes
                          : p.b ? p.b + (int64_t)g * p.N * kbytes : p.b_ptrs[g];
    b += j0 * E;
    const int nk = (int)((contr + Tn::kRows - 1) / Tn::kRows);

    // K-major A: pieces of 8 rows, 128 bytes of each; turned operands: pieces of kPieceRows rows
    const int c16 = ((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7)) * 16;
    auto issue = [&](int s) {
      char *st = lds + (s % M::kStages) * M::kStageBytes;
      const int64_t first = (int64_t)s * Tn::kRows;
      const int left = s < nk ? (int)min64(Tn::kRows, contr - first) : 0;  // contraction values of the stage
      auto turned = [&](const char *base, int64_t ld, int width, char *to) {
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            (void *)gemm::uniform_ptr(base + (left > 0 ? first * ld : 0)), (short)0, (int)(max(left, 1) * ld), 0x00020000);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int u = wave + q * M::kWaves, row = u * Tn::kPieceRows + lane / Tn::kSlots;
          const int c = Tn::slot(row, lane % Tn::kSlots) * 16;  // its own inverse
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              r, (GL_LDS void *)(to + u * 1024), 16,
              row < left && c < width * E ? (uint32_t)(row * (int)ld + c) : kPastEnd, 0, 0, 0);
        }
      };
      if constexpr (WGRAD) {
        turned(a, nbytes, rows, st);
      } else {
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void *)gemm::uniform_ptr(a), (short)0,
                                                                           (int)(rows * nbytes), 0x00020000);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int u = wave + q * M::kWaves;
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              r, (GL_LDS void *)(st + u * 1024), 16,
              c16 < left * E ? (uint32_t)((8 * u + (lane >> 3)) * (int)nbytes + c16) : kPastEnd,
              left > 0 ? (int)(first * E) : 0, 0, 0);
        }
      }
      turned(b, kbytes, cols, st + TILE * 128);
    };
    const int blocks = (rows - wm * 16 + 31) / 32;
    f32x4_t acc[2][M::kBlocks];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < M::kBlocks; ++i) acc[h][i] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < M::kStages - 1; ++s) issue(s);
    for (int s = 0; s < nk; ++s) {
      __builtin_amdgcn_sched_barrier(0);
      gemm::wait_vm<(M::kStages - 2) * M::kPieces>();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      issue(s + M::kStages - 1);
      const char *st = lds + (s % M::kStages) * M::kStageBytes;
      i32x4_t fb[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) fb[h][c] = Tn::frag(st + TILE * 128, wn * 32 + h * 16, c, lane);
#pragma unroll
      for (int i = 0; i < M::kBlocks; ++i) {
        if (i >= blocks) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          i32x4_t fa;
          if constexpr (WGRAD) {
            fa = Tn::frag(st, i * 32 + wm * 16, c, lane);
          } else {
            const int r = i * 32 + wm * 16 + fr;
            fa = *(const i32x4_t *)(st + r * 128 + (((4 * c + fq) ^ ((r >> 1) & 7)) << 4));
          }
          acc[0][i] = Op::mma(fb[0][c], fa, acc[0][i]);
          acc[1][i] = Op::mma(fb[1][c], fa, acc[1][i]);
        }
      }
    }
    void *out = WGRAD && !p.out ? p.out_ptrs[g] : p.out;
    const int64_t out0 = WGRAD ? (p.out ? (int64_t)g * p.N * p.K : 0) + i0 * p.K : (g_off + i0) * p.K;
#pragma unroll
    for (int i = 0; i < M::kBlocks; ++i) {
      const int rl = i * 32 + wm * 16 + fr;
      if (rl >= rows) break;
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
        put4<EL>(out, at, v);
      }
    }
    gemm::wait_vm0();
    __syncthreads();
  }
}

template <int IN, int EL, bool WGRAD, int TILE>
inline hipError_t launch_glu_back_tile(const BackParams &p, hipStream_t s) {
  const int64_t tiles_j = (p.K + TILE - 1) / TILE, groups = p.T < p.G ? p.T : p.G;
  const int64_t items = WGRAD ? p.G * ((p.N + TILE - 1) / TILE) * tiles_j : ((p.T + TILE - 1) / TILE + groups) * tiles_j;
  hipLaunchKernelGGL((glu_back_kernel<IN, EL, WGRAD, TILE>), dim3((unsigned)(items < 8192 ? items : 8192)),
                     dim3(MidTile<TILE>::kThreads), 0, s, p);
  return hipGetLastError();
}

// Whether a product goes by the small tiles: fp32 always (the grouped calls' fp32 kernel works on the
// vector units: 4 groups, 333 rows, K 1024, F 1024, both products 386 us; here 81), and 16-bit types
// where 256 x 256 tiles are few.  Measured (us, bf16; tiles of 64 / 128 / 256):
//   dx by tiles of 256:   16 (1 group, 256 rows, K 2048 F 2048) 41 / 60 / 59     64 (4, 1024, 2048, 2048) 79 / 62 / 86
//                        132 (1, 8192, 1024, 1024) 92 / 73 / 49                  272 (64, 1024, 1024, 512) 42 / 43 / 31
//   dW  by tiles of 256: 128 (1, 2048, 2048, 2048) 104 / 79 / 189                512 (4, 1024, 2048, 2048) 96 / 72 / 176
//                        512 (1, 4096, 4096, 4096) 719 / 540 / 261              1024 (16, 1024, 2048, 1024) 112 / 89 / 56
// (between, the 256-row kernel cuts long groups' tiles into parts that meet in memory)
inline bool glu_back_small(const BackParams &p, bool wgrad) {
  const int64_t groups = p.T < p.G ? p.T : p.G, tj = (p.K + 255) / 256;
  if (!wgrad) return ((p.T + 255) / 256 + groups) * tj < 128;
  const int64_t tiles = groups * ((p.N + 255) / 256) * tj;
  return tiles < 512 || (tiles < 1024 && p.T / groups < 2048);
}

// Tiles of 128 where there are enough of them: dx 192 (4 groups, 1024 rows, K 2048 F 2048) 62 us, of
// 64 79; 144 (16, 256, 1024, 512) 16.3 and 13.7.  dW 128 (1, 8192, 1024, 1024) 140 and 104; 1024 (4,
// 1024, 2048, 2048) 72 and 96.  fp32 tiles of 128 are up to twice as slow and at most a tenth faster.
template <int IN, int EL>
inline hipError_t launch_glu_back(const BackParams &p, bool wgrad, bool out_f32, hipStream_t s) {
  if constexpr (IN == IN_F32) {
    return wgrad ? launch_glu_back_tile<IN, EL, true, 64>(p, s) : launch_glu_back_tile<IN, EL, false, 64>(p, s);
  } else {
    const int64_t groups = p.T < p.G ? p.T : p.G, tj = (p.K + 127) / 128;
    if (!wgrad) {
      if (((p.T + 127) / 128 + groups) * tj >= 192) return launch_glu_back_tile<IN, EL, false, 128>(p, s);
      return launch_glu_back_tile<IN, EL, false, 64>(p, s);
    }
    if (groups * ((p.N + 127) / 128) * tj >= 192)
      return out_f32 ? launch_glu_back_tile<IN, EL_F32, true, 128>(p, s) : launch_glu_back_tile<IN, EL, true, 128>(p, s);
    return out_f32 ? launch_glu_back_tile<IN, EL_F32, true, 64>(p, s) : launch_glu_back_tile<IN, EL, true, 64>(p, s);
  }
}

}  // namespace gl
