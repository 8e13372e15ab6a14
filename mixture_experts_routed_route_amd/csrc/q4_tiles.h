// How a product of many rows goes into tiles and launches: plain constant expressions,
// so that a host program can walk over them.
#pragma once

#include <cstdint>

namespace moe {

constexpr int kTileM = 128, kTileN = 256, kTileThreads = 256;

// A launch: `rows` rows of x from `row` on; `whole` tiles of kTileM rows first, then tiles
// of half as many rows, `tiles` in all; `grid` workgroups.
struct TileLaunch { int64_t row, rows; int whole, tiles; unsigned grid; };

// The launch from row `row` on, of M rows and tn tiles across. Tiles go in full rounds of
// the compute units' workgroups (two each), and one more round of half tiles where what is
// left fits it. A launch holds fewer than 2^32 threads: 2^23 tiles and a round.
constexpr TileLaunch tile_launch_at(int64_t row, int64_t M, int64_t tn, int ncu) {
  const int64_t most = (1 << 23) / tn > 1 ? (1 << 23) / tn : 1;   // rows of tiles
  const int64_t rows = M - row < most * kTileM ? M - row : most * kTileM;
  const int64_t down = (rows + kTileM - 1) / kTileM, slots = 2 * (int64_t)ncu;
  int64_t big = down * tn / slots * slots / tn;   // rows of tiles in full rounds
  const int64_t halves = (rows - big * kTileM + kTileM / 2 - 1) / (kTileM / 2);
  if (halves * tn > slots) big = down;
  const int64_t whole = big * tn, rest = big == down ? 0 : halves * tn;
  return {row, rows, (int)whole, (int)(whole + rest), (unsigned)((whole + 7) / 8 * 8 + (rest + 7) / 8 * 8)};
}

// The tile of workgroup n: its first row (of the launch) and column; rows 0 for none. An
// XCD's workgroups (numbers equal modulo 8) take neighbouring tiles, first of the whole
// ones, then of those of half the rows.
struct TileAt { int64_t row, column; int rows; };
__attribute__((always_inline)) constexpr TileAt tile_at(int n, int tiles_n, int whole, int tiles) {
  const int big = (whole + 7) & ~7;
  const bool all = n < big;
  const int k = all ? n : n - big, count = all ? whole : tiles - whole;
  const int per = (count + 7) / 8, local = (k & 7) * per + (k >> 3);
  if ((k >> 3) >= per || local >= count) return {0, 0, 0};
  const int64_t column = (int64_t)(local % tiles_n) * kTileN, down = local / tiles_n;
  if (all) return {down * kTileM, column, kTileM};
  return {(int64_t)(whole / tiles_n) * kTileM + down * (kTileM / 2), column, kTileM / 2};
}

}  // namespace moe
