// Which kernel a bf16 grouped product or weight gradient takes, by its sizes alone (not part of the ABI).
// Host code that needs nothing of HIP, so that the CPU tests can ask it too.
#pragma once

#include <stdint.h>

namespace moe {
namespace bf16 {

enum Epilogue { kPlain, kGated, kGatedBackward };

// 256 x 256, 128 x 128, 64 x 128 (gated: 64 x 256) and 32 x 128 tiles, rows of A by columns of y; the
// contraction split over a workgroup's waves, 16 rows by 16 and 32.
enum GemmTile { kSquare256, kSquare128, kRows64, kRows32, kSplit16, kSplit32 };

constexpr int kCus = 256;

// Times in us, "a | b" for a choice and the next one below, weights 4096 x 6144 each.
inline GemmTile gemm_tile(int E, int N, int64_t R, Epilogue epilogue, bool transposed) {
  const int64_t hit = R < E ? R : E;   // at most so many experts have rows
  const int64_t mean = hit > 0 ? R / hit : 0;
  // tiles of q rows by c columns, for groups of the mean size
  auto items = [&](int q, int c) { return hit * ((mean + q - 1) / q) * ((N + c - 1) / c); };
  // - 256 x 256 where groups have more than one 128-row chunk and the tiles are more than half of the CUs, one
  //   each: 16 groups of 160 rows 201 | 231 (transposed 161 | 243, gated 215 | 260), of 128 182 | 171 (144 | 145,
  //   190 | 206); 9 of 256: 144 tiles, 190 | 257; 17 of 256, 2048 x 2048: 136 tiles, 50 | 62, 8 of 512: 128 tiles,
  //   46 | 39; 24 of 384, 784 x 1048: 192 tiles, 31 | 25, of 512 35 | 44.
  if (mean > 128 && items(256, 256) > kCus / 2) return kSquare256;
  // - The contraction split over a workgroup's waves, 16 x 16 while that is one round of the CUs: one group
  //   of 16 rows 13.1 | 16.1, of 24 20.4 | 15.4; then 16 x 32 for one round, or two where several chunks
  //   share weights: one of 64 rows 27 | 39, of 96 39 | 40 (gated 28 | 54, 39 | 53); 8 of one row, 2048 x
  //   2048: 512 tiles of one chunk each, 16.4 | 13.7.
  if (!transposed && items(16, 16) <= kCus) return kSplit16;
  if (!transposed && items(16, 32) <= (mean > 16 ? 2 : 1) * kCus) return kSplit32;
  if (epilogue == kGated) return kRows64;
  // - 128 x 128 where 64 rows are not enough and there is more than one for each CU: 16 groups of 96 rows
  //   183 | 206, of 64 151 | 145; 8 of 256, 2048 x 2048: 256 tiles, 28 | 25, of 512: 512 tiles, 38 | 46.
  if (mean > 64 && items(128, 128) > kCus) return kSquare128;
  // - 32 x 128 for one round: one group of 128 rows 31 | 42 (transposed 32 | 45, backward 33 | 45), 8 of 64, 2048
  //   x 2048, 14.6 | 17.4; 8 of 32, 4096 x 2048, 21.8 | 22.1; two rounds, transposed: one of 512 rows 50 | 46.
  return items(32, 128) <= kCus ? kRows32 : kRows64;
}

// Whether a weight gradient takes 256 x 256 tiles (otherwise 128 x 128).  Large ones, one for each CU at a
// time, need a contraction that pays for their start and end, and enough tiles or enough of it that the last
// round counts little.  In us, large | small, D binary32: 16 groups of 384 rows, 4096 x 6144, 477 | 500, of 256
// 403 | 397; 8 of 1024, 2048 x 2048, 76 | 82, of 512 54 | 54 (bf16 46 | 41); one of 4096, 4096 x 6144, 207 |
// 230, of 1024 72 | 65; one of 4096, 2048 x 2048: 64 tiles, 92 | 53.
inline bool wgrad_large(int E, int N, int K, int64_t R) {
  const int64_t tiles = static_cast<int64_t>(E) * ((N + 255) / 256) * ((K + 255) / 256), mean = R / E;
  return mean >= 384 && tiles >= kCus * 3 / 4 && tiles * mean >= kCus * 2048;
}

}  // namespace bf16
}  // namespace moe
