// Which kernel takes a call of linear_fp8_block, its tile's rows of X and how many
// CTAs (pairs) cut K: arithmetic on sizes, for the host alone.  64 bits throughout,
// as K may hold 2^24 blocks of some hundred ns each.
#pragma once

#include <stdint.h>

namespace gbf {

constexpr int kBlockCols = 128;           // columns that share a scale (and rows, in a weight)
constexpr int64_t block_count(int64_t n) { return (n + kBlockCols - 1) / kBlockCols; }

constexpr int kLbMaxSplit = 8;            // single CTAs that cut K: a portable cluster
constexpr int kBpMaxSplit = 4;            // pairs that do
constexpr int kBpTile = 256;              // a pair's tile: rows of X, and channels

// What the kernels find on a GPU.
struct LinearBlockRoom {
  int sms;
  int clusters[kBpMaxSplit + 1];          // by split: clusters of that many pairs that fit at once (0: unknown)
};

struct LinearBlockPlan {
  int rows;                               // 16, 32, 64, 128: single CTAs; kBpTile: pairs
  int split;
  int64_t tiles;
};

inline int64_t linear_block_tiles(int64_t m, int64_t n, int rows) {
  const int64_t cols = rows == kBpTile ? kBpTile : kBlockCols;
  return (m + rows - 1) / rows * ((n + cols - 1) / cols);
}

// Single CTAs cut K while every one still has an SM to itself (the next call's may
// then come beside it) and keeps four blocks.
inline int linear_block_split(int64_t tiles, int64_t blocks, int sms) {
  int split = 1;
  while (split < kLbMaxSplit && tiles * split * 2 <= sms && blocks >= split * 2 * 4) split *= 2;
  return split;
}

// Pairs cut K while all tiles' clusters fit the GPU at once and each pair keeps six blocks.
inline int linear_block_pair_split(int64_t tiles, int64_t blocks, const LinearBlockRoom& room) {
  int split = kBpMaxSplit;
  while (split > 1 && (blocks < split * 6 || tiles > room.clusters[split])) --split;
  return split;
}

// About how long the single CTAs take with 64 or 128 rows, which with
// linear_block_pair_ns() decides who takes a call of more than 32 rows.
// Measured: a K block of a tile 270 or 335 ns, its start and end 2.2 us, joining
// a cluster's sums 1.5 or 3 us more.  The estimates against the measured times
// (us; 64 rows a tile, 128, pairs), N x K = 4096 x 4096: 128 rows 8.0 / 9.0, 7.9 /
// 9.1, 14.3 / 16; 512 rows 21.7 / 21.4, 12.9 / 13.3, 17.4 / 18; 1024 rows 43.4 / 46,
// 25.8 / 26, 19.7 / 19.3.  16384 x 4096, 256 rows: 43.4 / 44, 25.8 / 27.6, 19.7 / 21.9.
// 4096 x 11008, 333 rows: 50.8 / 47, 31.0 / 29.7, 28.0 / 28.0.
inline int64_t linear_block_ns(int64_t m, int64_t n, int64_t k, int rows, int sms) {
  const int64_t tiles = linear_block_tiles(m, n, rows), waves = (tiles + sms - 1) / sms, blocks = block_count(k);
  const int split = linear_block_split(tiles, blocks, sms);
  return waves * (2200 + (blocks + split - 1) / split * (rows == 64 ? 270 : 335)) + (split > 1 ? (rows == 64 ? 1500 : 3000) : 0);
}

// The same of pairs: a K block 390 ns, a tile's end 2.2 us, the call's start and end
// 5 us, joining a cluster's sums 4 us more.
inline int64_t linear_block_pair_ns(int64_t m, int64_t n, int64_t k, const LinearBlockRoom& room) {
  const int64_t tiles = linear_block_tiles(m, n, kBpTile), blocks = block_count(k);
  const int split = linear_block_pair_split(tiles, blocks, room);
  const int64_t fit = room.clusters[split];
  if (fit < 1) return INT64_MAX;
  return (tiles + fit - 1) / fit * ((blocks + split - 1) / split * 390 + 2200) + 5000 + (split > 1 ? 4000 : 0);
}

// Sizes as the entry point admits them (each below 2^31, fewer than 2^31 tiles of 64 x
// 128).  Up to 32 rows `room.clusters` is not read.
inline LinearBlockPlan plan_linear_block(int64_t m, int64_t n, int64_t k, const LinearBlockRoom& room) {
  LinearBlockPlan p;
  p.rows = m <= 16 ? 16 : 32;
  if (m > 32) {
    const int64_t t64 = linear_block_ns(m, n, k, 64, room.sms), t128 = linear_block_ns(m, n, k, 128, room.sms),
                  tp = linear_block_pair_ns(m, n, k, room);
    p.rows = tp < t64 && tp < t128 ? kBpTile : t64 <= t128 ? 64 : 128;
  }
  p.tiles = linear_block_tiles(m, n, p.rows);
  p.split = p.rows == kBpTile ? linear_block_pair_split(p.tiles, block_count(k), room)
                              : linear_block_split(p.tiles, block_count(k), room.sms);
  return p;
}

}  // namespace gbf
