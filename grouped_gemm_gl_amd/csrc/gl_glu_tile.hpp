// Grouped products with a gated or scaled epilogue on 256-row tiles, for groups of many rows.
//
// A workgroup of eight waves takes 256 rows of a group by two sets of 128 weight rows, B0 and
// B1: the gate's and the other half's rows of the same 128 columns (plain: 256 neighbouring
// columns).  So h_g and h_u of an output are in the same lane, and the epilogue is in registers.
// The contraction goes by stages of 128 bytes of every row (64 values of 16 bits, 128 of 8, 32
// of 32: the same kernel for each, but for the matrix instruction).  Waves are 4 x 2; a wave has
// two blocks of 16 rows, 64 rows apart, of each half of the tile's rows, A0 and A1, by 64 columns
// of each of B0 and B1 (so where blocks past the tile's last row are skipped, 64 rows are a quarter
// of the work for every wave).
//
// A stage is four phases, one quadrant of the wave's outputs each, and each phase reads half
// an operand from LDS, asks for half an operand of the stage after next, and multiplies:
//   phase   reads          loads          multiplies
//     0     A0(s)          B0(s+2)        A0 B0
//     1     B1(s)          A0(s+2)        A0 B1
//     2     A1(s)          B1(s+2)        A1 B1
//     3     B0(s+1)        A1(s+2)        A1 B0
// A half's place in LDS is asked for again one phase after it was read, and what is loaded is
// read seven phases later, so a wave has 12 to 14 loads of 1 KiB in flight all the time and
// waits (vmcnt) for none that is younger than six phases: 96-112 KiB a CU, nearly the whole
// ring of two stages, with no wait for a stage as a whole.
//
// The waves 4-7 run one barrier behind the waves 0-3, which share their SIMDs: while one of a
// SIMD's two waves multiplies, the other reads.  A wave's reads are complete (lgkmcnt) before the
// barrier that ends its reading, so the loads that the other group sends after it may write there.
//
// The pipeline runs on over tiles: the last two stages of a tile ask for the first two of the
// next, whose loads are under way during the epilogue.  So the tiles' places are
// found ahead, 64 at a time by the lanes of each wave, and kept in LDS: nothing in the loop loads from
// memory to registers, or waits for it.
//
// Addresses: every stream is a buffer resource on a half's first row whose length ends with the
// last valid row, so rows past the group's or the matrix's end load zeros without a test; a lane's
// offset from there is the same for every stream, because the rows of both operands have the same
// length; past the row's end (the last stage) lanes take an offset out of range, and get zeros.
//
// The products of the backward whose operands lie with the other index contiguous (dx's weights, both of
// dW's) stage them as they lie, contraction row after contraction row, and turn them on the way out of LDS
// (read_turned, which waits for itself: there a phase's loads go out before its reads).
//
// Bound by the matrix cores: 8 groups, 16384 rows, K 4096 F 7168 bf16 1425 us, 1350 TFLOP/s (with h 1475), int8
// 760-790 us, 2430-2530 TOP/s; a library product of that size reaches 1438 and 2313.  dx and dW 1640-1720 and
// 1660-1690 us, 1120-1170 and 1140-1160 TFLOP/s, by the number of their reads: a turned fragment is four reads where
// the others are two, and a phase waits for its own.  Matrix cores busy 70% and 59% of the CUs' cycles (83%
// forward, 80% the gradient), LDS 27% and 24% (34%, 32%), conflicts in 1% and 4% of those.  Without the lag of the
// second wave group 1651.
#pragma once

#include "gl_gemm_tile.hpp"
#include "gl_glu_choice.hpp"
#include "gl_glu_mid.hpp"

namespace gl {

constexpr int kTileWaves = 8, kTileThreads = 64 * kTileWaves;
constexpr int kTileRowsM = 256, kHalf = 128;
constexpr int kStageB = 128;                 // bytes of a row in a stage
constexpr int kHalfBytes = kHalf * kStageB;  // a half operand of a stage in LDS
constexpr int kRingBytes = 4 * kHalfBytes;   // A0, A1, B0, B1
constexpr uint32_t kOutside = 0x80000000u;   // past every resource's end

// 16 rows by 64 columns of a wave's part of an output between registers, where a lane has four
// columns of a row in each of four blocks, and memory, as whole lines: through the wave's own 2 KiB
// of LDS behind the ring, 128 bytes of a row at a time (all 64 columns of 16-bit values, 32 of
// 32-bit ones).  Stored straight from the registers, 16 rows by 32 bytes an instruction, the lines
// came together in L2 from quarters.  The 16-byte slots of a row are permuted by the row so that
// neither side's accesses meet in a bank.  Rows and columns outside go to an offset past the
// resource's end, which drops stores and loads zeros.
constexpr int kStoreBytes = 2048;
template <int EL>
struct TileStore {
  typedef typename Quad<EL>::raw raw_t;
  typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
  char *buf;
  int lane, row, rows, col;  // the piece's first row in the tile, rows of the tile, first column
  static constexpr int E = elem_bytes(EL), kBlocks = 8 / E, kPieces = 4 / kBlocks;
  __device__ __forceinline__ static int slot(int r, int s) { return (s ^ ((r >> 1) & 7)) << 4; }
  // the lane's four columns of block j of a piece
  __device__ __forceinline__ raw_t *quad(int j) const {
    const int r = lane & 15, q = lane >> 4;
    return (raw_t *)(buf + r * 128 + (E == 4 ? slot(r, 4 * j + q) : slot(r, 2 * j + (q >> 1)) + (q & 1) * 8));
  }
  // the lane's 16 bytes of move k: in LDS, and their offset from the tile's first row
  __device__ __forceinline__ u32x4_t *moved(int k) const {
    const int r = k * 8 + (lane >> 3);
    return (u32x4_t *)(buf + r * 128 + slot(r, lane & 7));
  }
  __device__ __forceinline__ uint32_t place(int s, int k, int64_t ld, int width) const {
    const int r = row + k * 8 + (lane >> 3), c = col + s * (128 / E) + (lane & 7) * (16 / E);
    return r < rows && c < width ? (uint32_t)((r * (int)ld + c) * E) : 0x80000000u;
  }
  __device__ __forceinline__ static void order() {  // lanes' accesses on either side stay there
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t block(const void *base, int64_t row0, int64_t ld, int64_t col0) const {
    return gemm::rsrc_at(gemm::uniform_ptr((const char *)base + (row0 * ld + col0) * E));
  }
  template <bool ONCE = false, class F>
  __device__ __forceinline__ void put(void *base, int64_t row0, int64_t ld, int64_t col0, int width, F value) const {
    const __amdgpu_buffer_rsrc_t rs = block(base, row0, ld, col0);
#pragma unroll
    for (int s = 0; s < kPieces; ++s) {
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) {
        *quad(j) = value(s * kBlocks + j);
        __builtin_amdgcn_sched_barrier(0);  // one value's registers at a time
      }
      order();
      const u32x4_t v0 = *moved(0), v1 = *moved(1);
      __builtin_amdgcn_raw_buffer_store_b128(v0, rs, place(s, 0, ld, width), 0, ONCE ? 2 : 0);
      __builtin_amdgcn_raw_buffer_store_b128(v1, rs, place(s, 1, ld, width), 0, ONCE ? 2 : 0);
      order();
    }
  }
  __device__ __forceinline__ void get(const void *base, int64_t row0, int64_t ld, int64_t col0, int width,
                                      raw_t (&out)[4]) const {
    const __amdgpu_buffer_rsrc_t rs = block(base, row0, ld, col0);
#pragma unroll
    for (int s = 0; s < kPieces; ++s) {
      const u32x4_t v0 = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, place(s, 0, ld, width), 0, 0));
      const u32x4_t v1 = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, place(s, 1, ld, width), 0, 0));
      *moved(0) = v0;
      *moved(1) = v1;
      order();
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) out[s * kBlocks + j] = *quad(j);
      order();
    }
  }
};

constexpr int kPlacesBytes = 64 * 16;  // places of a wave's next 64 tiles

struct TilePlace {
  int g, jt;
  int rows;      // of the tile, 1 .. 256
  int64_t row0;  // the first in the packed rows; dW: of the group's
  int from, len;  // dW: the contraction, the group's rows
};

// ACT: a run-time activation would be three copies of the epilogue, whose common values the
// compiler computes ahead of them all and spills.
// RAGGED: row blocks past a tile's rows are neither read from LDS nor multiplied, which costs full
// tiles a tenth of their speed in branches.  kRaggedOnce: and the weights are loaded as data that is
// read once.  kWrittenOnce: full tiles whose outputs are stored as data that is not read soon.
template <int IN, int EL, int EPI, int ACT, int RAGGED>
__global__ __launch_bounds__(kTileThreads, 2) void glu_tile_kernel(GluParams p) {
  using Op = Operand<IN>;
  using acc_t = typename Op::acc_t;
  constexpr bool kTurnA = EPI == EPI_DW, kTurnB = EPI == EPI_DW || EPI == EPI_DX;
  constexpr bool kGated = EPI == EPI_GLU || EPI == EPI_GLU_GRAD;
  constexpr int kColsB = kGated ? kHalf : 2 * kHalf;  // output columns of a tile
  constexpr int kStageRows = kStageB / in_bytes(IN);  // contraction values of a stage
  using Tn = Turned<IN, kHalf>;
  constexpr bool kSkip = RAGGED == kRaggedTiles || RAGGED == kRaggedOnce;
  __shared__ __attribute__((aligned(1024))) char lds[2 * kRingBytes + kTileWaves * (kStoreBytes + kPlacesBytes)];

  const WsView ws = ws_view(p.ws, p.G);
  if (!ws_usable(ws.hdr, p.G, p.T)) return;
  const int64_t *__restrict__ off = ws.off;
  const int32_t *__restrict__ pre = ws.pre[tile_rows_index(kTileRowsM)];
  const int tiles_j = (int)((p.F + kColsB - 1) / kColsB);
  const int tiles_i = EPI == EPI_DW ? (int)((p.N + kTileRowsM - 1) / kTileRowsM) : 0;
  const int total = EPI == EPI_DW ? p.G * tiles_i * tiles_j : pre[p.G] * tiles_j;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int grid = gridDim.x, b = blockIdx.x;
  // each XCD (blockIdx % 8) walks a run of neighbouring tiles
  const int first = (grid & 7) == 0 ? (b & 7) * (grid >> 3) + (b >> 3) : b;
  if (first >= total) return;
  const int count = (total - first + grid - 1) / grid;  // tiles of this workgroup
  const int kb = (int)((EPI == EPI_DW ? p.N : p.K) * in_bytes(IN));  // bytes of a row of A
  const int fb_ = (int)(p.F * in_bytes(IN));                         // of a turned B
  // stages of a tile (two at least: loads are two stages ahead)
  auto stages_of = [&](int len) { return max(2, EPI == EPI_DW ? (len + kStageRows - 1) / kStageRows : (kb + kStageB - 1) / kStageB); };

  // ---- places of 64 tiles, found one a lane, in LDS: (group, first row, tile indices, contraction)
  int base = 0;
  int4 *const places = (int4 *)(lds + 2 * kRingBytes + kTileWaves * kStoreBytes + wave * kPlacesBytes);
  auto fill = [&]() {
    const int w = first + min(base + lane, count - 1) * grid;
    int lo = 0, local, mt;
    if constexpr (EPI == EPI_DW) {
      const int per = tiles_i * tiles_j;
      lo = w / per;
      local = w - lo * per;
      mt = tiles_i;
    } else {
      const int q = w / tiles_j;
      int hi = p.G;  // the last g with pre[g] <= q
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= q) lo = mid;
        else hi = mid;
      }
      local = w - pre[lo] * tiles_j;
      mt = pre[lo + 1] - pre[lo];
    }
    // bands of kOrdN column tiles, in a band blocks of kOrdM row tiles, row tiles fastest
    const int cb = local / (mt * gemm::kOrdN), bw = min(gemm::kOrdN, tiles_j - cb * gemm::kOrdN);
    const int l2 = local - cb * mt * gemm::kOrdN;
    const int rb = l2 / (gemm::kOrdM * bw), bh = min(gemm::kOrdM, mt - rb * gemm::kOrdM);
    const int l3 = l2 - rb * gemm::kOrdM * bw;
    const int it = rb * gemm::kOrdM + l3 % bh, jt = cb * gemm::kOrdN + l3 / bh;
    int4 e;
    e.x = lo;
    bool good;
    if constexpr (EPI == EPI_DW) {  // the group's first row; both tile indices; the group's rows
      e.y = (int)off[lo];
      e.z = (jt << 13) | it;
      e.w = (int)(off[lo + 1] - off[lo]);
      good = e.w >= 0 && e.y >= 0 && (int64_t)e.y + e.w <= p.T && it < tiles_i && jt < tiles_j;
    } else {  // the tile's first row; its column and rows
      const int64_t r0 = off[lo] + (int64_t)it * kTileRowsM;
      const int rows = (int)min64(kTileRowsM, off[lo + 1] - r0);
      e.y = (int)r0;
      e.z = (jt << 9) | rows;
      e.w = 0;
      good = mt > 0 && local >= 0 && it < mt && jt < tiles_j && rows > 0 && r0 >= 0 && r0 + rows <= p.T;
    }
    // a failed check: a tile without rows, of which nothing is stored; dW's has the matrix's rows, and -1 of the
    // contraction says so
    if (GL_DEVICE_CHECKS && !device_check(good, p.ws)) e = make_int4(0, 0, 0, EPI == EPI_DW ? -1 : 0);
    places[lane] = e;
    TileStore<EL>::order();
  };
  fill();
  auto place = [&](int n) {  // of the workgroup's n-th tile
    // (as asm: the compiler would wait for all loads to LDS that are under way)
    i32x4_t v;
    asm volatile("ds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(v)
                 : "v"((uint32_t)(uintptr_t)(GL_LDS int4 *)(places + (n - base)))
                 : "memory");
    const int4 e = make_int4(v[0], v[1], v[2], v[3]);
    TilePlace t;
    t.g = __builtin_amdgcn_readfirstlane(e.x);
    const int first_row = __builtin_amdgcn_readfirstlane(e.y), jr = __builtin_amdgcn_readfirstlane(e.z);
    if constexpr (EPI == EPI_DW) {
      t.from = first_row;
      t.jt = jr >> 13;
      t.row0 = (int64_t)(jr & 8191) * kTileRowsM;
      t.rows = (int)min64(kTileRowsM, p.N - t.row0);
      t.len = __builtin_amdgcn_readfirstlane(e.w);
    } else {
      t.from = t.len = 0;
      t.row0 = first_row;
      t.jt = jr >> 9;
      t.rows = jr & 511;
    }
    return t;
  };

  // ---- loads: pieces of 1 KiB, wave w has the pieces w and w + 8 of each half: 8 rows by 128 bytes,
  // of a turned operand 4 contraction rows by 256
  const int c16 = ((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7)) * 16;  // place in the stage's 128 bytes
  const uint32_t voff = (uint32_t)(8 * wave + (lane >> 3)) * (uint32_t)kb + (uint32_t)c16;
  const int trow = 4 * wave + (lane >> 4), tc16 = Tn::slot(trow, lane & 15) * 16;  // rows 32 apart: the same slots
  const uint32_t tva = (uint32_t)(trow * kb + tc16), tvb = (uint32_t)(trow * fb_ + tc16);
  __amdgpu_buffer_rsrc_t ra, rb0, rb1;
  const char *ta = nullptr, *tb = nullptr;  // turned operands: the tile's first column of the stage's first row
  int wide_a = 0, wide_b = 0;               // and bytes of columns
  int load_tile = 0, load_stage = 0, load_nk = 2, load_len = 0;  // what the next four phases ask for
  auto rsrc = [&](const char *at, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)gemm::uniform_ptr(at), (short)0, bytes, 0x00020000);
  };
  auto aim = [&]() {  // the streams of tile load_tile
    if (load_tile >= count) return;
    asm volatile("" ::: "memory");  // the place is read here alone, not ahead of the test in every stage
    const TilePlace t = place(load_tile);
    const int64_t col0 = (int64_t)t.jt * kColsB, left = p.F - col0;
    load_nk = stages_of(t.len);
    if constexpr (EPI == EPI_DW) {
      load_len = t.len;
      ta = p.x + (int64_t)t.from * kb + t.row0 * in_bytes(IN);
      wide_a = t.rows * in_bytes(IN);
      tb = p.w + (int64_t)t.from * fb_ + col0 * in_bytes(IN);
      wide_b = (int)min64(2 * kHalf, left) * in_bytes(IN);
      return;
    }
    const char *wg = group_weights<IN, EPI>(p, t.g);
    ra = rsrc(p.x + t.row0 * kb, (GL_DEVICE_CHECKS ? max(t.rows, 1) : t.rows) * kb);
    if constexpr (EPI == EPI_DX) {
      load_len = (int)p.K;
      tb = wg + col0 * in_bytes(IN);
      wide_b = (int)min64(2 * kHalf, left) * in_bytes(IN);
      return;
    }
    rb0 = rsrc(wg + col0 * kb, (int)min64(kHalf, left) * kb);
    if (EPI == EPI_PLAIN)
      rb1 = left > kHalf ? rsrc(wg + (col0 + kHalf) * kb, (int)min64(kHalf, left - kHalf) * kb) : rsrc(wg + col0 * kb, kb);
    else
      rb1 = rsrc(wg + (p.F + col0) * kb, (int)min64(kHalf, left) * kb);
  };
  // half 0 A0, 1 A1, 2 B0, 3 B1 of stage load_stage into ring slot `ring`
  auto issue = [&](auto half_tag, int ring) __attribute__((always_inline)) {
    constexpr int half = decltype(half_tag)::value;
    char *to = lds + ring * kRingBytes + half * kHalfBytes + wave * 1024;
    if constexpr (half < 2 ? kTurnA : kTurnB) {
      const int ld = half < 2 ? kb : fb_, wide = half < 2 ? wide_a : wide_b;
      const int left = __builtin_amdgcn_readfirstlane(  // rows of the stage
          load_tile < count ? min(kStageRows, load_len - load_stage * kStageRows) : 0);
      const __amdgpu_buffer_rsrc_t r = rsrc(half < 2 ? ta : tb, max(left, 0) * ld);
      constexpr int c = (half & 1) * (kHalf * in_bytes(IN));  // the half's first column
      const uint32_t v = half < 2 ? tva : tvb;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (GL_LDS void *)(to + q * 8192), 16,
                                                 tc16 + c < wide ? v + (uint32_t)(32 * q * ld + c) : kOutside, 0, 0,
                                                 RAGGED == kRaggedOnce && half >= 2 ? 2 : 0);
    } else {
      const int at = load_stage * kStageB;
      const int lim = load_tile < count ? kb - at : 0;  // bytes of the row left
      const __amdgpu_buffer_rsrc_t r = half < 2 ? ra : half == 2 ? rb0 : rb1;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t o = voff + (uint32_t)(((half == 1) * kHalf + q * 64) * kb);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (GL_LDS void *)(to + q * 8192), 16, c16 < lim ? o : kOutside,
                                                 lim > 0 ? at : 0, 0, RAGGED == kRaggedOnce && half >= 2 ? 2 : 0);
      }
    }
  };
  auto next_stage = [&]() {
    if (kTurnA) ta += (int64_t)kStageRows * kb;
    if (kTurnB) tb += (int64_t)kStageRows * fb_;
    if (++load_stage == load_nk) {
      load_stage = 0;
      ++load_tile;
      aim();
    }
  };

  // ---- fragments: 16 bytes of row l % 16 of a block, of the stage's half s (turned: of column l % 16)
  const int fr = lane & 15, fq = lane >> 4;
  // places of the first block of A and of B in a half: the others and the other half of the stage are
  // an offset or a bit away
  const uint32_t at_a = kTurnA ? Tn::place(wm * 16, lane) : (wm * 16 + fr) * kStageB + ((fq ^ (fr >> 1)) & 7) * 16;
  const uint32_t at_b = kTurnB ? Tn::place(wn * 64, lane) : (wn * 64 + fr) * kStageB + ((fq ^ (fr >> 1)) & 7) * 16;
  auto opaque = [](uint32_t v) {
    if (kTurnB) asm volatile("" : "+v"(v));  // found at each read (kept, they are the registers that spill)
    return v;
  };
  const uint32_t lds0 = (uint32_t)(uintptr_t)(GL_LDS char *)lds;
  i32x4_t fa[2][2], fb[2][4][2];  // [block][half of the stage]; two sets of B
  int blocks = 4;  // row blocks of the wave that hold rows: (A half, i) in turn are 64 rows apart
  auto read_a = [&](int half, int ring) {
    const uint32_t o = opaque(at_a + ring * kRingBytes + half * kHalfBytes);
    if constexpr (kTurnA) {
      const uint32_t at[2] = {lds0 + o, lds0 + (o ^ 128)};
      read_turned<256>(at, fa);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (!kSkip || 2 * half + i < blocks)
#pragma unroll
          for (int s = 0; s < 2; ++s) fa[i][s] = *(const i32x4_t *)(lds + (o ^ (64 * s)) + i * 64 * kStageB);
    }
  };
  auto read_b = [&](int set, int half, int ring) {
    const uint32_t o = opaque(at_b + ring * kRingBytes + half * kHalfBytes);
    if constexpr (kTurnB) {
      const uint32_t at[4] = {lds0 + o, lds0 + (o ^ 32), lds0 + (o ^ 64), lds0 + (o ^ 96)};
      read_turned<256>(at, fb[set]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) fb[set][j][s] = *(const i32x4_t *)(lds + (o ^ (64 * s)) + j * 16 * kStageB);
    }
  };
  acc_t acc[2][2][2][4];  // [A half][B half][row block][column block]
  auto zero = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int l = 0; l < 4; ++l) acc[i][j][k][l] = acc_t{0, 0, 0, 0};
  };
  auto multiply = [&](int set, int half, acc_t(&c)[2][4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (!kSkip || 2 * half + i < blocks)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) c[i][j] = Op::mma(fb[set][j][s], fa[i][s], c[i][j]);
  };
  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
  auto barrier = [&] {
    fence();
    __builtin_amdgcn_s_barrier();
    fence();
  };
  auto read_done = [&]() {  // ends a phase's reading: own reads back, loads of six phases ago there
    fence();
    __builtin_amdgcn_s_waitcnt(0x007c);  // vmcnt(12) lgkmcnt(0)
    barrier();
  };
  // One stage in ring slot `ring`, B0 in register set S on entry, the next stage's B0 in the
  // other set after it.
  auto stage = [&](auto set_tag, int ring) __attribute__((always_inline)) {
    constexpr int S = decltype(set_tag)::value;
    // (a turned operand's reads wait for themselves: the phase's loads go out before them)
    auto phase = [&](auto load_tag, bool last, auto read, bool turned) __attribute__((always_inline)) {
      if (!turned) read();
      issue(load_tag, ring);
      if (last) next_stage();
      if (turned) read();
      read_done();
    };
    phase(std::integral_constant<int, 2>{}, false, [&] { read_a(0, ring); }, kTurnA);
    multiply(S, 0, acc[0][0]);
    barrier();
    phase(std::integral_constant<int, 0>{}, false, [&] { read_b(1 - S, 3, ring); }, kTurnB);
    multiply(1 - S, 0, acc[0][1]);
    barrier();
    phase(std::integral_constant<int, 3>{}, false, [&] { read_a(1, ring); }, kTurnA);
    multiply(1 - S, 1, acc[1][1]);
    barrier();
    phase(std::integral_constant<int, 1>{}, true, [&] { read_b(1 - S, 2, ring ^ 1); }, kTurnB);
    multiply(S, 1, acc[1][0]);
    barrier();
  };

  // ---- the first two stages
  aim();
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    issue(std::integral_constant<int, 2>{}, s);
    issue(std::integral_constant<int, 0>{}, s);
    issue(std::integral_constant<int, 3>{}, s);
    issue(std::integral_constant<int, 1>{}, s);
    next_stage();
  }
  fence();
  gemm::wait_vm<12>();
  barrier();

  int ring = 0;
  for (int n = 0; n < count; ++n) {
    zero();
    const TilePlace t = place(n);
    blocks = (t.rows - wm * 16 + 63) / 64;
    const int nk = stages_of(t.len);
    // B0 of the first stage (again: the last tile's last stage read it, but held through the
    // epilogue it would cost 32 registers), by all waves before the first loads may replace it
    read_b(0, 2, ring);
    gemm::wait_lgkm0();
    barrier();
    if (wave >= 4) barrier();  // one barrier behind
    int k = 0;
    for (; k + 1 < nk; k += 2) {
      stage(std::integral_constant<int, 0>{}, ring);
      stage(std::integral_constant<int, 1>{}, ring ^ 1);
    }
    if (k < nk) {
      stage(std::integral_constant<int, 0>{}, ring);
      ring ^= 1;
    }
    if (wave < 4) barrier();  // in step again: both groups' epilogues at the same time

    // the lane index, opaque here, so that nothing of the epilogue's addresses is kept in registers
    // through the stages
    int le = lane;
    asm volatile("" : "+v"(le));
    const int er = le & 15, eq = le >> 4;
    const int64_t col0 = (int64_t)t.jt * kColsB;
    const int width = (int)min64(kHalf, p.F - col0);  // columns of the first set
    const int width1 = kGated ? width : (int)min64(kHalf, p.F - col0 - kHalf);
    const int64_t second = kGated ? p.F + col0 : col0 + kHalf;  // the second set's first column
    ColumnTerms<IN, EL> ct[2][4];
    RowScale rs[2][2];
    if constexpr (!kTurnB) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = wn * 64 + j * 16 + eq * 4;  // a lane past the last column takes the last four, and is not stored
        ct[0][j] = column_terms<IN, EL, EPI>(p, t.g, col0 + min(c, width - 4));
        ct[1][j] = column_terms<IN, EL, EPI>(p, t.g, width1 > 0 ? second + min(c, width1 - 4) : col0);
      }
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (IN == IN_I8) rs[a][i] = RowScale(p.x_scale[t.row0 + min(a * kHalf + i * 64 + wm * 16 + er, max(t.rows, 1) - 1)]);
    }
    // dW is the group's own matrix; with accumulate, a group without rows is not touched
    void *const out = EPI == EPI_DW ? p.out ? (char *)p.out + (int64_t)t.g * p.N * p.F * elem_bytes(EL) : p.out_ptrs[t.g] : p.out;
    const bool untouched = EPI == EPI_DW && ((p.accumulate && t.len == 0) || (GL_DEVICE_CHECKS && t.len < 0));
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        typedef Quad<EL> Q;
        const TileStore<EL> st{lds + 2 * kRingBytes + wave * kStoreBytes, le, a * kHalf + i * 64 + wm * 16, t.rows, wn * 64};
        if (2 * a + i >= blocks || untouched) continue;
        auto value = [&](int b, int j) { return finish<IN, EL>(acc[a][b][i][j], rs[a][i], ct[b][j]); };
        auto gate = [&](int j) { return Q::pack(value(0, j)); };
        auto other = [&](int j) { return Q::pack(value(1, j)); };
        if constexpr (kTurnB) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (b == 1 && width1 <= 0) break;
            typename Q::raw old[4];
            if (EPI == EPI_DW && p.accumulate) st.get(out, t.row0, p.F, b ? second : col0, b ? width1 : width, old);
            st.template put<RAGGED == kWrittenOnce>(out, t.row0, p.F, b ? second : col0, b ? width1 : width, [&](int j) {
              const acc_t v = acc[a][b][i][j];
              float4 o = make_float4(v[0], v[1], v[2], v[3]);
              if (EPI == EPI_DW && p.accumulate) {
                const float4 m = Q::value(old[j]);
                o = make_float4(o.x + m.x, o.y + m.y, o.z + m.z, o.w + m.w);
              }
              return Q::pack(o);
            });
          }
        } else if constexpr (EPI == EPI_PLAIN) {
          st.put(p.out, t.row0, p.F, col0, width, gate);
          if (width1 > 0) st.put(p.out, t.row0, p.F, second, width1, other);
        } else if constexpr (EPI == EPI_GLU) {
          st.put(p.out, t.row0, p.F, col0, width, [&](int j) {
            float4 none;
            return Q::pack(mul4(activate4<false, ACT>(value(0, j), none), value(1, j)));
          });
          if (p.h) {
            st.put(p.h, t.row0, 2 * p.F, col0, width, gate);
            st.put(p.h, t.row0, 2 * p.F, second, width, other);
          }
        } else {
          typename Q::raw da[4], out[4];  // da, then da h_u act'(h_g); the forward's output
          st.get(p.da, t.row0, p.F, col0, width, da);
          st.put(p.out, t.row0, 2 * p.F, second, width, [&](int j) {
            float4 slope;
            const float4 y = activate4<true, ACT>(value(0, j), slope), u = value(1, j), d = Q::value(da[j]);
            da[j] = Q::pack(mul4(mul4(d, u), slope));
            out[j] = Q::pack(mul4(y, u));
            return Q::pack(mul4(d, y));
          });
          if (p.a) st.put(p.a, t.row0, p.F, col0, width, [&](int j) { return out[j]; });
          st.put(p.out, t.row0, 2 * p.F, col0, width, [&](int j) { return da[j]; });
        }
      }
    if (n + 3 - base >= 64) {  // the loads are at most two tiles ahead
      base = n + 1;
      fill();
    }
  }
  gemm::wait_vm0();  // no load may be under way to the LDS of a workgroup that has ended
}

template <int IN, int EL, int EPI, int ACT>
inline hipError_t launch_glu_tile(const GluParams &p, int64_t items, int ragged, hipStream_t s) {
  const dim3 grid(gemm::persistent_grid(items)), block(kTileThreads);
  if constexpr (IN == IN_I8 || EPI == EPI_DX) {
    if (ragged == kRaggedOnce) {
      hipLaunchKernelGGL((glu_tile_kernel<IN, EL, EPI, ACT, kRaggedOnce>), grid, block, 0, s, p);
      return hipGetLastError();
    }
  }
  if constexpr (EPI == EPI_DW) {
    if (ragged == kWrittenOnce) {
      hipLaunchKernelGGL((glu_tile_kernel<IN, EL, EPI, ACT, kWrittenOnce>), grid, block, 0, s, p);
      return hipGetLastError();
    }
  } else {
    if (ragged) {
      hipLaunchKernelGGL((glu_tile_kernel<IN, EL, EPI, ACT, kRaggedTiles>), grid, block, 0, s, p);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((glu_tile_kernel<IN, EL, EPI, ACT, kFullTiles>), grid, block, 0, s, p);
  return hipGetLastError();
}

// The instances of choose_glu (gl_glu_choice.hpp).
template <int IN, int EL, int EPI>
inline hipError_t launch_glu(const GluParams &p, hipStream_t s) {
  const GluChoice c = choose_glu(IN, EPI == EPI_PLAIN, p.G, p.T, p.K, p.F);
  if constexpr (IN == IN_F32)
    if (c.kernel == GluChoice::kFew) return launch_glu_few<EPI>(p, s);
  if (c.kernel == GluChoice::kMid) {
    if constexpr (IN == IN_F32) {
      if (c.parts == 2) return launch_glu_mid<IN, EL, EPI, 32, 64, 2>(p, false, s);
      return c.rows == 32 ? launch_glu_mid<IN, EL, EPI, 32, 64>(p, c.once, s)
                          : launch_glu_mid<IN, EL, EPI, 64, 64>(p, c.once, s);
    } else {
      if (c.rows == 128) return launch_glu_mid<IN, EL, EPI, 128, 128>(p, c.once, s);
      if constexpr (IN == IN_I8)
        return c.parts == 2 ? launch_glu_mid<IN, EL, EPI, 32, 64, 2>(p, false, s)
                            : launch_glu_mid<IN, EL, EPI, 32, 64>(p, c.once, s);
      else if (c.parts == 2) return launch_glu_mid<IN, EL, EPI, 32, 32, 2>(p, false, s);
      else if (c.rows == 32) return launch_glu_mid<IN, EL, EPI, 32, 32>(p, c.once, s);
      else return launch_glu_mid<IN, EL, EPI, 64, 64>(p, c.once, s);
    }
  }
  if constexpr (EPI != EPI_PLAIN) {
    if (p.act == ACT_GELU) return launch_glu_tile<IN, EL, EPI, ACT_GELU>(p, c.items, c.ragged, s);
    if (p.act == ACT_GELU_TANH) return launch_glu_tile<IN, EL, EPI, ACT_GELU_TANH>(p, c.items, c.ragged, s);
  }
  return launch_glu_tile<IN, EL, EPI, ACT_SILU>(p, c.items, c.ragged, s);
}

}  // namespace gl
