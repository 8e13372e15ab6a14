// Walks over the launches and tiles of products of many rows: every launch within what
// one may hold, every element of the output in exactly one tile.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <vector>

#include "q4_tiles.h"

using namespace moe;

#define CHECK(cond, ...)                 \
  do {                                   \
    if (!(cond)) {                       \
      std::printf(__VA_ARGS__);          \
      std::printf("  [%s]\n", #cond);    \
      std::exit(1);                      \
    }                                    \
  } while (0)

static void launches(int64_t M, int64_t N, int ncu) {
  const int64_t tn = (N + kTileN - 1) / kTileN;
  int64_t row = 0;
  while (row < M) {
    const TileLaunch t = tile_launch_at(row, M, tn, ncu);
    CHECK(t.row == row && t.rows > 0 && t.rows <= M - row, "%lld x %lld", (long long)M, (long long)N);
    CHECK((uint64_t)t.grid * kTileThreads < (1ull << 32), "%lld x %lld: %u workgroups", (long long)M, (long long)N, t.grid);
    CHECK(t.whole >= 0 && t.tiles >= t.whole && t.grid >= (unsigned)t.tiles, "%lld x %lld", (long long)M, (long long)N);
    // rows that whole tiles and halves cover
    const int64_t big = t.whole / tn * kTileM, half = (t.tiles - t.whole) / tn * (kTileM / 2);
    CHECK(t.whole % tn == 0 && (t.tiles - t.whole) % tn == 0, "%lld x %lld", (long long)M, (long long)N);
    CHECK(big + half >= t.rows, "%lld x %lld: %lld rows of %lld", (long long)M, (long long)N, (long long)(big + half),
          (long long)t.rows);
    CHECK(row + t.rows == M || t.rows % kTileM == 0, "%lld x %lld", (long long)M, (long long)N);
    row += t.rows;
  }
}

static void cover(int64_t M, int64_t N, int ncu) {
  const int64_t tn = (N + kTileN - 1) / kTileN;
  const TileLaunch t = tile_launch_at(0, M, tn, ncu);
  CHECK(t.rows == M, "%lld rows in one launch", (long long)M);
  std::vector<int> seen((size_t)((M + 63) / 64 * tn), 0);   // 64 rows x a tile's columns
  for (unsigned n = 0; n < t.grid; ++n) {
    const TileAt a = tile_at((int)n, (int)tn, t.whole, t.tiles);
    for (int r = 0; r < a.rows; r += 64)
      if (a.row + r < M) ++seen[(size_t)((a.row + r) / 64 * tn + a.column / kTileN)];
  }
  for (int v : seen) CHECK(v == 1, "%lld x %lld on %d units: a tile %d times", (long long)M, (long long)N, ncu, v);
}

int main() {
  const int64_t most = (1ll << 31) - 1, wide = 1ll << 26;
  for (int64_t M : {most, most - 126, most - 127, most - 1000, (int64_t)1 << 30, (int64_t)70000, (int64_t)17})
    for (int64_t N : {(int64_t)1, (int64_t)256, (int64_t)257, (int64_t)4096, (int64_t)31000, (int64_t)1050000, wide})
      for (int ncu : {256, 304, 32, 1})
        if (M * ((N + 255) / 256) < (1ll << 40)) launches(M, N, ncu);
  for (int64_t M = 17; M < 6000; M += 1 + M / 9)
    for (int64_t N : {1, 255, 256, 257, 1000, 4096, 5000, 50000})
      for (int ncu : {256, 7}) cover(M, N, ncu);
  std::printf("ok\n");
  return 0;
}
