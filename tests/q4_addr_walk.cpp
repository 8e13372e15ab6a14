// Walks over every load that the products of few rows, the tiles and the layer for a
// few tokens make of 4-bit weights, by the offsets that the kernels use: each word read
// lies inside the operand, though the descriptor's check counts only a lane's own
// offset, and each value that is used is read from its place.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "q4_addr.h"

using namespace moe;

static long long g_loads = 0;

#define CHECK(cond, ...)                 \
  do {                                   \
    if (!(cond)) {                       \
      std::printf(__VA_ARGS__);          \
      std::printf("  [%s]\n", #cond);    \
      std::exit(1);                      \
    }                                    \
  } while (0)

struct Operand {
  const char* what;
  long long bytes;    // of all rows
  long long base;     // of the strip's first row
  uint32_t range;     // of the strip's descriptor
};

// words of a load, each read if its own offset lies in the descriptor's range
static void read(const Operand& o, LoadAt at, int words) {
  ++g_loads;
  for (int i = 0; i < words; ++i) {
    const uint64_t v = (uint64_t)at.v + 4u * i;
    if (v + 4 > o.range) continue;
    const long long a = o.base + (long long)v + at.s;
    CHECK(a >= 0 && a + 4 <= o.bytes, "%s: word at %lld of %lld", o.what, a, o.bytes);
  }
}
// bytes from `want` of the operand on are read by the load's first ones
static void used(const Operand& o, LoadAt at, long long want, int bytes) {
  CHECK((uint64_t)at.v + bytes <= o.range, "%s: %d used bytes at %u behind the range %u", o.what, bytes, at.v, o.range);
  CHECK(o.base + (long long)at.v + at.s == want, "%s: reads %lld, not %lld", o.what, o.base + (long long)at.v + at.s, want);
}

// group, bytes of parameters, and whether rows may hold an odd number of 2-byte scales
struct Format { int group, pb; };

static void strip(const Format& f, long long N, long long n0, int K, int strip_rows, bool whole, bool runs) {
  const int blocks = (K + 127) / 128;
  const uint32_t rb = K / 2, pb = K / f.group * f.pb, per = 128 / f.group * f.pb;
  const uint32_t rows = N - n0 < strip_rows ? N - n0 : strip_rows;
  const Operand q{"codes", N * rb, n0 * rb, rows * rb}, p{"parameters", N * pb, n0 * pb, rows * pb};
  for (int kb = 0; kb < blocks; ++kb) {
    for (uint32_t lane = 0; lane < 64; ++lane) {
      const uint32_t r = lane >> 2, piece = lane & 3;
      const LoadAt c = codes_at(codes_start(lane, rb), kb, whole);
      read(q, c, 4);
      if (r < rows && kb * 128 + (int)piece * 32 < K)
        used(q, c, (n0 + r) * rb + kb * 64 + piece * 16, 16);
      if (pb % 4 == 0 && !runs) {
        const LoadAt a = params_at(params_start(lane, pb), kb, per, whole);
        read(p, a, per / 4);
        if (lane < rows) {
          const int left = (K - kb * 128 + f.group - 1) / f.group * f.pb;   // to the row's end
          used(p, a, (n0 + lane) * pb + (long long)kb * per, left < (int)per ? left : per);
        }
      }
      if (pb % 4 == 0 && runs) {   // a run may start at any block
        const LoadAt a = run_at(run_start(lane, pb), kb, per);
        read(p, a, 4);
        const long long at = (long long)kb * per + piece * 16;   // of the row
        if (r < rows && at < pb) used(p, a, (n0 + r) * pb + at, pb - at < 16 ? pb - at : 16);
      }
    }
  }
}

// The second launch of the layer: strips of 16 rows whose parameters come for two
// blocks at once, and of 8 rows where lanes of the upper half have the next block.
static void down(const Format& f, long long N, long long n0, int K) {
  const int blocks = K / 128;
  const uint32_t rb = K / 2, pb = K / f.group * f.pb, per = 128 / f.group * f.pb;
  const Operand q16{"codes", N * rb, n0 * rb, 16 * rb}, p16{"parameters", N * pb, n0 * pb, 16 * pb};
  const Operand q8{"codes of 8 rows", N * rb, n0 * rb, 8 * rb}, p8{"parameters of 8 rows", N * pb, n0 * pb, 8 * pb};
  for (int kb = 0; kb < blocks; kb += 2)
    for (uint32_t lane = 0; lane < 64; ++lane) {
      read(q16, codes_at(codes_start(lane, rb), kb, true), 4);
      if (per == 8) {
        const LoadAt a = run_at(params_start(lane, pb), kb, per);
        read(p16, a, 4);
        if (lane < 16) used(p16, a, (n0 + lane) * pb + (long long)kb * per, kb + 1 < blocks ? 16 : 8);
      }
      const bool odd = kb + 1 >= blocks;
      uint32_t vq = codes_start(lane, rb), vp = params_start(lane, pb);
      if (lane >= 32) vq = odd ? kPastEnd : vq - 8 * rb + 64;
      if (lane >= 8 && lane < 16) vp = odd ? kPastEnd : vp - 8 * pb + per;
      read(q8, codes_at(vq, kb, true), 4);
      read(p8, params_at(vp, kb, per, true), per / 4);
      if (!(lane >= 32 && odd))
        used(q8, codes_at(vq, kb, true), (n0 + (lane >> 2) % 8) * rb + (kb + (lane >= 32)) * 64 + (lane & 3) * 16, 16);
    }
}

int main() {
  const Format formats[3] = {{32, 2}, {32, 4}, {64, 4}};
  const int Ks[] = {32, 64, 96, 128, 160, 192, 256, 288, 448, 640, 1024, 1056, 1088, 1152, 2048, 2080, 4096, 4128, 14336};
  const long long Ns[] = {1, 7, 15, 16, 17, 31, 33, 77, 100, 1001, 4096};
  for (const Format& f : formats)
    for (int K : Ks) {
      if (K % f.group) continue;
      for (long long N : Ns) {
        const long long last = (N - 1) / 16 * 16;
        for (long long n0 : {0ll, last}) {
          strip(f, N, n0, K, 16, false, false);   // tiles; rows of an odd number of scales
          strip(f, N, n0, K, 16, false, true);
          if (K % 128 == 0) strip(f, N, n0, K, 16, true, true);
        }
      }
      if (K % 128 == 0)
        for (long long n0 : {0ll, 128ll, 240ll, 248ll})
          if (n0 + 16 <= 256) down(f, 256, n0, K);
      if (K % 128 == 0) down(f, 128, 112, K);
    }
  // the largest offsets stay below the lanes that read nothing
  CHECK(codes_at(codes_start(63, 1u << 21), (1 << 15) - 1, false).v < kPastEnd, "long rows");
  CHECK(run_at(run_start(63, (1u << 22) / 8), (1 << 15) - 1, 16).v < kPastEnd, "long rows");
  CHECK(run_at(kPastEnd, (1 << 15) - 1, 16).v >= kPastEnd && codes_at(kPastEnd, (1 << 15) - 1, false).v >= kPastEnd, "no load");
  std::printf("ok %lld loads\n", g_loads);
  return 0;
}
