// Internal declarations of the 8-bit block format, its products and layer,
// and the norms around a block.
#pragma once

#include "moe_internal.h"

namespace moe {

// Compute units of the current device (moe_api.hip).
moe_status current_cus(int* ncu);

// ---- 8-bit blocks (quant_f8.hip, gemm_f8.hip) ------------------------------
// Codes [rows, K] and scales [rows, ceil(K / 128)] of rows; codes [mats, N, K]
// and scales [mats, ceil(N / 128), ceil(K / 128)] of weights.
hipError_t launch_quant_rows(const void* x, int dt, int64_t rows, int K,
                             void* q, float* s, hipStream_t st);
hipError_t launch_quant_weights(const void* w, int dt, int64_t mats, int N,
                                int K, void* q, float* s, hipStream_t st);

// A layer's first launch: x's rows quantised, the plan's groups listed.
enum F8Meta : int32_t { kF8Parts = 0, kF8Tiles = 1, kF8MetaCount = 2 };
struct F8PrepareArgs {
  const void* x; int xdt; int T, D;
  uint8_t* q; float* s;
  const int32_t* counts; const int32_t* offsets; int n_exp;
  int thin_rows;            // experts of up to so many rows: parts
  int32_t* parts;           // (expert, row0, rows <= 16, first pair)
  int32_t* tiles;           // (expert, row0) tiles of kFullBM rows
  int32_t* meta;            // [kF8MetaCount] their numbers
};
hipError_t launch_f8_prepare(const F8PrepareArgs& a, hipStream_t st);

// One product on e4m3 rows: out[row, n] = sum_b As[row, b] Bs[n / 128, b]
// sum_{k in block b} A[row, k] B[n, k].
struct F8Args {
  int mode;                 // 0: plain, rows 0 .. M; 1: gate/up with SwiGLU
                            // over a plan's pairs, x's rows gathered; 2: down
                            // over a plan's pairs, rows in pair order
  int64_t M;                // mode 0: rows; on the tile split into
  int tiles256;             // ... this many tiles of 256 rows, then
  int tail_tiles, tail_rows;// tiles of tail_rows (128 or 64)
  int K, N;                 // reduction; output width (gate/up: features)
  const uint8_t* A;         // [rows, K] codes, or (strips over a plan, groups
                            // of at most lds_rows rows) values of type adt
  const float* As;          // [rows, ceil(K / 128)]
  int adt, lds_rows;        // adt MOE_F8B128: codes and scales
  const uint8_t* B0; const float* B0s;   // weights and their block scales
  const uint8_t* B1; const float* B1s;   // gate/up: W_up
  const int32_t* pair_token;
  const int32_t* offsets;   // [n_exp + 1]
  const int32_t* list;      // strip and stream: (expert, row0, rows, first
                            // pair) groups of at most 16 rows; tile: (expert,
                            // row0)
  const int32_t* groups;    // device: the list's length
  int max_groups;           // most groups the list can hold
  void* out; int odt;       // plain and down: [rows, N]; gate/up: strip f32
                            // [P, N], stream and tile codes [P, N] ...
  float* out_s;             // ... with scales [P, N / 128]
  float clamp;
};
hipError_t launch_f8_strip(const F8Args& a, int ncu, hipStream_t s);
// modes 1 and 2 over a plan's parts
hipError_t launch_f8_stream(const F8Args& a, hipStream_t s);
// whether strips may take groups of `rows` rows of K values unquantised
bool f8_strip_raw_fits(int rows, int K);
// list: (expert, row0) tiles of kFullBM rows, max_groups of them at most.
// prec 0 (modes 0 and 2): codes in the 8-bit matrix unit; 1: widened to f16
hipError_t launch_f8_tile(const F8Args& a, int prec, hipStream_t s);

// One-token calls on MOE_F8B128 weights (gemv_f8.hip).
struct F8OneArgs {
  const void* x; int xdt;   // [D]
  const uint8_t* wg; const uint8_t* wu; const uint8_t* wd;
  const float* wgs; const float* wus; const float* wds;
  const int32_t* ids;       // [k] the token's experts (plan)
  const int32_t* tok2pair;  // [k] their pair rows, -1 if dropped
  const int32_t* offsets;   // [E + n_shared + 1]
  const float* w;           // [k] routing weights
  float* h;                 // [P, F] SwiGLU outputs
  void* y; int ydt;         // [D]
  int D, F, k, E, n_shared;
  float clamp;
};
bool f8_one_fits(int D, int F, int k, int n_shared);
hipError_t launch_f8_one_gateup(const F8OneArgs& a, hipStream_t s);
hipError_t launch_f8_one_down(const F8OneArgs& a, hipStream_t s);

// The layer on MOE_F8B128 weights (api_f8.hip): its device workspace and its
// launches, on a plan's arrays.
struct F8Plan {
  moe_plan_desc desc;
  const int32_t* ids; const float* w; const int32_t* tok2pair;
  const int32_t* counts; const int32_t* offsets; const int32_t* pair_token;
  bool decode;              // at most kDecodeT tokens: the plan's group list
  const int32_t* dlist; const int32_t* dmeta;
};
struct F8Layer {
  const void* x; int xdt;
  const void* wg; const float* wgs;
  const void* wu; const float* wus;
  const void* wd; const float* wds;
  int D, F, ncu;
  void* y; int ydt;
  char* ws;
  moe_options o;
};
size_t f8_layer_bytes(const moe_plan_desc& d, int D, int F);
// steps of the layer in order; `phase` is the index moe_phase_times reports
constexpr int kF8Steps = 6;
int f8_step_phase(int step);
hipError_t launch_f8_step(const F8Plan& p, const F8Layer& l, int step, hipStream_t s);

// ---- norms (norm.hip) --------------------------------------------------------
struct NormArgs {
  int T, D, nb;             // nb: blocks of 128 values a row
  int rdt, udt, xdt, wdt, gdt;
  int gate_token;           // 1: g has a value per token, 0: per channel
  int unit;                 // 1: w and p stand for 1 + w, 1 + p
  float alpha, eps;
  const void* r; const void* u; const void* p; const void* g; const void* w;
  void* r_out; void* x; float* xs;
};
hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s);

struct NormBwdArgs {
  int T, D;
  int rdt, udt, dxdt, wdt, gdt, gate_token, unit;
  float alpha, eps;
  const void* r; const void* u; const void* p; const void* g; const void* w;
  const void* dr; const void* dx;
  void* dr_out; void* du;
  float* dw; float* dp; float* dg_channel; float* dg_token;
  float* part;              // norm_backward_part_floats
};
size_t norm_backward_part_floats(int T, int D);
hipError_t launch_norm_backward(const NormBwdArgs& a, hipStream_t s);

}  // namespace moe
