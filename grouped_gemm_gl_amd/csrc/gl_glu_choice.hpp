// Which kernel and tile a gated or scaled grouped product, and the products of its backward, run on: rules
// on types and sizes.  Plain C++, so that a test on the host can ask for the choice too.
#pragma once

#include <cstdint>

namespace gl {

// operand types
enum { IN_BF16 = 0, IN_F32 = 1, IN_F16 = 2, IN_I8 = 3 };
constexpr int in_bytes(int in) { return in == IN_F32 ? 4 : in == IN_I8 ? 1 : 2; }

// forms of the 256-row tiles (gl_glu_tile.hpp)
enum { kFullTiles = 0, kRaggedTiles = 1, kRaggedOnce = 2, kWrittenOnce = 3 };
constexpr int64_t kLastLevelCache = (int64_t)256 << 20;

struct GluChoice {
  enum Kernel { kFew, kMid, kTile } kernel;
  int rows, weight_rows, parts;  // kMid: the tile, parts of the contraction
  bool once;                     // kMid: the weights are loaded as data that is read once
  int ragged;                    // kTile: the form
  int64_t items;                 // kTile: the most tiles there can be
};

// Which kernel, by the rows of a group that has any (on average: the splits are on the device) and
// the most tiles there can be.  The tiles of 256 rows multiply at the rate of the matrix cores, those
// of 128 and 64 are enough for the chip in smaller problems and waste less on groups of few rows.
// Measured (us; 64 / 128 / 256 rows):
//   by rows a group, K 4096 F 7168, 8 groups, bf16:    16 rows 183 / 195 / 196   32 rows 217 / 189 / 208
//                                                     128 rows 418 / 250 / 254  512 rows 1350 / 656 / 444
//     (128 rows from 24 on: int8, small / 128: 64 of 1600, K 1408 N 2048 36.7 / 40.2, 64 of 4096 55 / 48.7, 4 of 130,
//     K 4096 N 14336 49 / 40; bf16 64 of 1600, K 2048 F 768 81 / 89, 8 of 256, K 4096 F 4096 134 / 105)
//   by tiles, one group, K 4096 F 4096: 512 rows (96 tiles of 256) 66 / 39 / 70   1024 (160) 130 / 76 / 71
//     K 1024 F 1024: 512 rows (80 tiles of 128, 24 of 256) 8.8 / 12.8 / 23        2048 (272, 72) 19 / 15 / 25
//   fp32, 32 cycles a matrix instruction: what counts is that no CU waits for another's tile.
//     4 groups, 333 rows, K 1024 F 2048 37 / 69 / 216;  8 groups, 16384 rows, K 4096 F 7168
//     (4032 tiles of 256) 16504 / 14747 / 14029
//     (Few rows on many wide experts lose by it: 64 of 64 rows, K 2048 F 7168 706 on tiles of 64 with weights read
//     once, 782 on those of 256; 64 of 2048 1662 / 1850; 64 of 4096, K 2048 F 4096 1497 / 1709.)
//   8-bit integers, 25 to 96 rows a group and weights past the cache, 128 / 256: 64 groups, K 2048 F 1408, 28 rows
//     78 / 69, 64 rows 89 / 80, 90 rows 105 / 86;  128 groups, K 2048 F 768 85 / 73, 102 / 89, 120 / 107;  8 groups,
//     K 4096 F 7168 102 / 100, 115 / 106, 129 / 117, but at 48 rows 102 / 109;  16 groups, K 4096 F 4096 111 / 119,
//     130 / 122, 132 / 155.
// Among the small tiles (rows by weight rows; us):
//   16 bits, 64 x 64 / 32 x 32: at most 256 tiles of 64: 2 groups, 64 rows, K 4096 F 2048 23.6 / 15.8, one of
//     300, K 1024 F 1024 8.3 / 7.6 (at 1 of 128, K 4096 F 4096, 384 tiles, 23.2 / 25.8).  At most 8 rows
//     a group: 64 of 256, K 4096 F 768 170 / 134, 8 of 16, K 4096 F 7168 156 / 136, but K 2048 72 / 76 and 81 / 84
//     (64 of 1024, K 2048 F 768 76 / 86).
//   8-bit integers, 64 x 64 / 32 x 64: 64 of 32 rows, K 1408 N 2048 16.1 / 13.5; 64 of 1024 37.8 / 34.4; one of
//     512, K 2048 N 1024 8.6 / 7.7; one of 32, K 4096 N 4096 10.8 / 11.2.
//   fp32, 64 x 64 / 32 x 64: up to 896 tiles of 32, for which 768 are under way at once: 8 of 600, K 2048 F 1024
//     (864) 71 / 60, but 4 of 333, K 1024 F 2048 (960) 37 / 41.  64 of 64, K 1024 F 512 39 / 34; one of 256,
//     K 4096 F 4096 (1152) 137 / 165.  4 of 333 rows, 780 / 900 / 990 / 1200 tiles: K 1024 37 / 32, 38 / 38, 38 / 43,
//     58 / 49;  K 4096 135 / 109, 135 / 131, 137 / 169, 212 / 185.
//   The contraction in one / two parts, by tiles of 32 x 64: 16 bits (on 32 x 32) 216 (8 of 64 groups, 8 rows, K 2048
//     F 768) 11.2 / 10.4, 96 (one of 64, K 2048 F 1024) 9.1 / 7.7, 256 (2 of 64, K 4096 F 2048) 16.0 / 17.5;  8-bit
//     integers 128 (one of 32, K 4096 N 4096) 11.1 / 8.6, 320 (8 of 64, K 2048 N 2048) 7.9 / 7.1, 1056 (64 of 32, K 1408
//     N 2048) 13.5 / 19.3;  fp32 320 (8 of 40, K 2048 F 1024) 35 / 26, 544 (one of 512, K 1024 F 1024) 24.6 / 28.0.
//     (8 groups of 64 rows, 16 bits, 190 / 220 / 260 / 320 tiles: K 1024 7.0 / 6.1, 7.1 / 6.2, 7.1 / 6.2, 7.5 / 6.5;
//     K 2048 11.0 / 10.4, 11.3 / 11.4, 12.2 / 11.9, 13.9 / 13.3;  K 4096 18.5 / 18.8, 18.9 / 19.2, 21.3 / 20.7, 24.0 /
//     22.7;  fp32, 4 of 333 rows, K 1024, 240 / 300 / 390 tiles 16.7 / 14.7, 22.9 / 27.3, 23.8 / 28.0.)
//     Weights of so few tiles are past the cache only where K is very long: they are not marked as read once.
// Weights of more than the 256 MB of the last-level cache that about one row tile of each group reads
// are loaded as data that is read once: 64 groups, 4099 rows, K 2048 F 1400, fp16 (734 MB of weights),
// tiles of 128 180 -> 172; with it 8-bit integers of F 1408 take 84 on tiles of 256, 95 on those of 128.
// Smaller ones lose what the cache holds from call to call (8 of 64 groups of 6 MB: 14.3 -> 16.5), and
// weights that more row tiles read lose it within the call (8 groups, 2048 rows, K 4096 F 7168 int8
// 89 -> 103).
// And fp32, at most 16 rows with few columns, by tiles of 64 weight rows (us; the contraction split over waves /
// tiles of 32 rows): 64 (4 groups, 8 rows, K 1024 F 512) 9.1 / 13.6, 192 (8 of 8, K 2048 F 768) 15.5 / 24.5, 256
// (16 of 64, K 1024 F 512) 14.4 / 16.1, 512 (8 of 8, K 2048 F 2048) 36.6 / 30.6.
// (8 groups of 256 rows, K 4096 F 7168, bf16: 297 us skipping what is past the rows, 306 not; of 512: 472 and 460)
inline GluChoice choose_glu(int in, bool plain, int64_t G, int64_t T, int64_t K, int64_t F) {
  const int64_t groups = T < G ? T : G, rows = T / groups, wide = (plain ? 1 : 2) * F;  // weight rows
  auto tiles = [&](int64_t r) { return ((T + r - 1) / r + groups) * ((wide + r - 1) / r); };
  auto mid = [](int r, int w, int parts, bool once) { return GluChoice{GluChoice::kMid, r, w, parts, once, 0, 0}; };
  if (in == IN_F32 && T <= 16 && groups * ((wide + 63) / 64) <= 256) return {GluChoice::kFew, 0, 0, 1, false, 0, 0};
  const bool once = rows <= 96 && groups * wide * K * in_bytes(in) > kLastLevelCache;
  const bool large = in == IN_F32  ? tiles(256) >= 2048
                     : in == IN_I8 ? tiles(256) >= 160 && (rows > 96 || (rows > 24 && once))
                                   : tiles(256) >= 160 && rows > 96;
  if (large)  // (fp32 has no form of its own for weights that are read once)
    return {GluChoice::kTile, 256, 256, 1, false, once && in == IN_I8 ? kRaggedOnce : rows <= 256 ? kRaggedTiles : kFullTiles,
            tiles(256)};
  const int64_t tiles32 = ((T + 31) / 32 + groups) * ((wide + 63) / 64);
  if (in == IN_F32) {
    if (tiles32 <= 384) return mid(32, 64, 2, false);
    return rows <= 32 || tiles32 <= 896 ? mid(32, 64, 1, once) : mid(64, 64, 1, once);
  }
  if (rows > 24 && tiles(128) >= 256) return mid(128, 128, 1, once);
  if (in == IN_I8) return tiles32 <= 384 ? mid(32, 64, 2, false) : mid(32, 64, 1, once);
  if (tiles32 <= 224) return mid(32, 32, 2, false);
  return rows <= 8 || tiles(64) <= 256 ? mid(32, 32, 1, once) : mid(64, 64, 1, once);
}

struct BackChoice {
  int rows, cols, parts;  // the tile (256: gl_glu_tile.hpp's), parts of the contraction
  bool once;              // below 256: dx's weights or dW are past the cache
  int tiles;              // 256: the form
  int64_t items;
};

// Which tiles.  fp32: dW those of 64 (of 128 up to twice as slow, at most a tenth faster) with a ring of
// three, three workgroups a CU, because a group's rows are few stages (4 groups, 333 rows, K 1024 F 1024
// 34.4 us with a ring of four, 30.3 of three; one of 4096 rows 167 and 169); dx 32 x 64 up to 896 of them, for
// which 768 are under way at once (47 us on tiles of 64, 32 on these; one of 4096 rows, 2064 of them, 153 and
// 165), up to 384 with the contraction in two parts (240: those 32 -> 27; 864: 66 -> 84).  (The grouped calls' fp32 kernel works on the vector units: both products 386 us, here 57.)
// 16 bits, dx: up to 256 tiles of 32 x 64 those, in two parts (144: one group, 256 rows, K 1024 F 1024 13.3 us
// on tiles of 64, 11.8 in one part, 9.7 in two; 544: 2 of 1024 rows 35.8 and 37.8 with dW), and else as
// measured for bf16 (us; tiles of 64 / 128 / 256), (groups, rows, K, F):
//   dx by tiles of 256:  16 (1, 256, 2048, 2048) 25 / 41 / 88     64 (4, 1024, 2048, 2048) 50 / 41 / 87
//                       144 (2, 4096, 2048, 2048) 116 / 89 / 89  272 (1, 4096, 4096, 4096) 439 / 318 / 220
//      and rows a group: 16 (64, 1024, 1024, 512) 36 / 34 / 27    64 (64, 4096, 2048, 768) 119 / 103 / 130
//      by tiles of 128: 144 (16, 256, 1024, 512) 9.9 / 11.9      192 (4, 1024, 2048, 2048) 50 / 41
//   dW by tiles of 256:  32 (1, 8192, 1024, 1024) 81 / 92 / 196  128 (1, 2048, 2048, 2048) 75 / 59 / 63
//                       256 (16, 256, 1024, 512) 32 / 25 / 17   1024 (16, 1024, 2048, 1024) 107 / 87 / 44
// What passes the last-level cache's 256 MB does not stay there: weights that one or two row tiles a group read
// and weight gradients then go past it (64 groups, 4099 rows, K 2048 F 1400 fp16, 734 MB each: dx 211 -> 172,
// dW 213 -> 185; 8 of 1024, K 4096 F 7168 dx 331 -> 282, dW 280 -> 262;
// fp32, 8 of 16, K 4096 F 4096 dx 223 -> 156, dW 333 -> 298).  Smaller weight gradients are left
// where their next reader finds them, though they too are written faster (1 of 512, K 2048 F 2048, 17 MB,
// 27.4 -> 25.8).
inline BackChoice choose_glu_back(int in, bool wgrad, bool out_f32, int64_t G, int64_t T, int64_t K, int64_t N) {
  const int64_t groups = T < G ? T : G, rows = T / groups;
  const int64_t tiles32 = ((T + 31) / 32 + groups) * ((K + 63) / 64);
  auto tile = [](int r, int c, int parts, bool once) { return BackChoice{r, c, parts, once, 0, 0}; };
  if (in == IN_F32) {
    if (wgrad) return tile(64, 64, 1, G * N * K * 4 > kLastLevelCache);
    if (tiles32 <= 384) return tile(32, 64, 2, false);
    const bool once = rows <= 96 && groups * K * N * 4 > kLastLevelCache;
    return rows <= 32 || tiles32 <= 896 ? tile(32, 64, 1, once) : tile(64, 64, 1, once);
  }
  auto tiles = [&](int64_t r) {
    return (wgrad ? groups * ((N + r - 1) / r) : (T + r - 1) / r + groups) * ((K + r - 1) / r);
  };
  if (!wgrad) {
    const bool large = groups * K * N * in_bytes(in) > kLastLevelCache;  // weights
    if (tiles(256) >= 160 && (rows <= 24 || rows > 96))
      return {256, 256, 1, false, rows > 256 ? kFullTiles : large ? kRaggedOnce : kRaggedTiles, tiles(256)};
    if (tiles(128) >= 192) return tile(128, 128, 1, large && rows <= 96);
    return tiles32 <= 256 ? tile(32, 64, 2, false) : tile(64, 64, 1, false);
  }
  if (tiles(256) >= 128)
    return {256, 256, 1, false, G * N * K * (out_f32 ? 4 : in_bytes(in)) > kLastLevelCache ? kWrittenOnce : kFullTiles,
            G * ((N + 255) / 256) * ((K + 255) / 256)};
  return tiles(128) >= 192 ? tile(128, 128, 1, false) : tile(64, 64, 1, false);
}

}  // namespace gl
