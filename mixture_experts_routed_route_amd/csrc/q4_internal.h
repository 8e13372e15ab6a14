// Internal declarations of the 4-bit quantiser, products on 4-bit weights and
// the layer for a few tokens.
#pragma once

#include <cmath>

#include "moe_internal.h"

namespace moe {

// Bytes of LDS a workgroup may use.
constexpr size_t kLdsBytes = 160 * 1024;

// Values of K that a workgroup's x takes in LDS at once: all (up to a multiple of
// 128), or the most that fit beside `other` bytes; one and two blocks take b1 and
// b2 bytes.
inline int lds_turn(size_t b1, size_t b2, size_t other, int K) {
  const int64_t all = ((int64_t)K + 127) / 128;
  const int64_t fit = 1 + (int64_t)((kLdsBytes - other - b1) / (b2 - b1));
  return (int)(128 * (all < fit ? all : fit));
}

// ---- quantiser (quant_q4.hip) ----------------------------------------------
// values [rows, K] of type dt to codes [rows, K / 2] and parameters of a 4-bit
// format; K a multiple of its group.
hipError_t launch_quant_q4(const void* w, int dt, int fmt, int64_t rows, int64_t K, void* data,
                           void* params, hipStream_t s);

// ---- products (gemm_q4.hip) --------------------------------------------------
// out[M, N] = x[M, K] . w[N, K]^T; fmt a 4-bit format
struct RowsArgs {
  const void* x; int xdt;
  const void* w; const void* params; int fmt;
  int64_t M; int N, K;
  void* out; int odt;
};
// up to 16 rows
hipError_t launch_rows_product(const RowsArgs& a, int ncu, hipStream_t s);
// any number of rows, 4-bit weights (gemm_q4_tile.hip)
hipError_t launch_q4_tile(const RowsArgs& a, int ncu, hipStream_t s);

// ---- the layer for a few tokens (decode.hip) -----------------------------------
constexpr int kFewT = MOE_DECODE_MAX_T;
struct FewArgs {
  const void* x; int xdt;            // [T, D]
  const float* logits;               // [T, E]
  const void* wg; const void* wu; const void* wd;     // [E + n_shared, ..]
  const void* wgs; const void* wus; const void* wds;  // 4-bit parameters, or null
  int fmt;                           // 4-bit format, or -1: weights in x's type
  int T, D, F, E, k, n_shared;
  int limit;                         // most pairs an expert keeps (T: all)
  float clamp;
  int parts;                         // h's 16-bit parts (few_hold), its power of two and that back
  float up, down;
  // workspace
  void* h;                           // [pairs, parts, F] SwiGLU outputs by expert
  float* w;                          // [T, E] routing weights of chosen experts
  int32_t* list;                     // [1 + 3 slots]: their number, experts, token masks, pairs before
  void* y; int ydt;                  // [T, D]
};
// experts that tokens can choose, and the shared one
constexpr int few_slots(int T, int E, int k, int n_shared) {
  const int64_t n = (int64_t)T * k;
  return (int)(n < E ? n : E) + n_shared;
}
// How h, the SwiGLU's f32 output, is held as an operand of the 16-bit matrix units.
//  * Three bf16 parts: 24 bits, f32's range. Beside bf16 weights, and beside 4-bit ones
//    whose layer has no limit.
//  * Two fp16 parts of h * up, the second one * kRestUp as well: 23 bits of what lies above
//    2^-14 / up, and 2^-37 / up in absolute terms below. A limit c bounds h by max(c, 0.28)
//    c (silu is above -0.28), and up brings that bound to 2^15: with the default of 7, 2^9.
//    Without (c^2 of 2^15 and more) up is 1, beside fp16 weights only: past 65504 h is
//    infinite there, as moe_forward's 16-bit h.
// Parts of 16 bits in all (two of bf16) put 1 output of bf16 in 300 to its neighbour.
constexpr float kRestUp = 4096.f;
struct FewHold { int parts; float up, down; };
inline FewHold few_hold(int xdt, int fmt, float clamp) {
  const float bound = (clamp > 0.28f ? clamp : 0.28f) * clamp;
  const bool bounded = clamp > 0.f && bound < 32768.f;
  if (fmt < 0 && xdt == MOE_BF16) return {3, 1.f, 1.f};
  if (!bounded) return {fmt < 0 ? 2 : 3, 1.f, 1.f};
  int e;
  std::frexp(bound, &e);   // bound < 2^e
  e = 15 - e < 100 ? 15 - e : 100;
  return {2, std::ldexp(1.f, e), std::ldexp(1.f, -e)};
}
// the most parts that any limit asks for
constexpr int few_max_parts(int xdt, int fmt) { return fmt >= 0 || xdt == MOE_BF16 ? 3 : 2; }
hipError_t launch_few_router(const void* x, int xdt, const void* w, float* logits, int T, int D, int E,
                             hipStream_t s);
hipError_t launch_few_gateup(const FewArgs& a, int ncu, hipStream_t s);
hipError_t launch_few_down(const FewArgs& a, int ncu, hipStream_t s);

}  // namespace moe
