// The whole layer for 1 to 16 tokens, from router logits to y, in two launches
// on gfx950 (moe_decode): no plan, no pair list, nothing between workgroups but
// the launch boundary.
//
//  * gate/up: every workgroup routes all tokens itself (a wave a token, k rounds of
//    a wave-wide maximum; the first one writes the routing for the second launch),
//    then its waves take (expert, 16 features) items: the expert's 16 gate and 16 up
//    rows against all tokens' rows of x at once, which lie in LDS (rows16.h). A token
//    that did not choose the expert costs no memory, only lanes of a matrix
//    instruction. h is kept in 16-bit parts that together hold its f32 bits
//    (FewH): the matrix units wait for memory anyway.
//  * down: a workgroup takes 8 or 16 output columns and all experts that were chosen,
//    in turns of as many as LDS holds h of, its waves taking runs of blocks of 128 of
//    F; each block's sums are scaled by the routing weights in f32 and added, the
//    waves' sums meet in LDS, y is rounded once. Sums run in a fixed order: the same
//    bits every time.
// The router's map, where asked for, is a launch before them.
//
// Bound by the chosen experts' weights, read once. Of D 2048, F 768, 16-bit, k 8 and a
// shared one of 128: one token 19 + 9 us (57 and 28 MB, 3 TB/s: about 8 and 4 us are
// launch, routing and latency), sixteen 102 + 63 us (5.1 and 4.2 TB/s). Of D 4096, F 2048,
// 4-bit with scales, 8 of 256: one token 24 + 13 us (3.2 and 2.9 TB/s), eight 125 + 88 us
// (4.3 and 3.1 TB/s; widening and scaling the codes is about half of that). Medians under
// the profiler, three sets of inputs in turn.
#include "rows16.h"
#include "route_key.h"
#include "q4_internal.h"

namespace moe {

namespace {

// the largest of a value over the wave, as a scalar
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#define MOE_MAX_STEP(CTRL, ROWS) \
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROWS, 0xF, false))
  MOE_MAX_STEP(0xB1, 0xF);    // quad_perm [1, 0, 3, 2]
  MOE_MAX_STEP(0x4E, 0xF);    // quad_perm [2, 3, 0, 1]
  MOE_MAX_STEP(0x141, 0xF);   // row_half_mirror
  MOE_MAX_STEP(0x140, 0xF);   // row_mirror
  MOE_MAX_STEP(0x142, 0xA);   // row_bcast:15 into rows 1, 3
  MOE_MAX_STEP(0x143, 0xC);   // row_bcast:31 into rows 2, 3
#undef MOE_MAX_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_sum_f(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Router's map: logits[t, e] = x[t] . w[e], a workgroup an expert, a slice of 8 values
// of the row a thread, f32 products in a fixed order. NT >= T.
template <class S, int NT>
__global__ __launch_bounds__(512) void few_router_kernel(const S* __restrict__ x, const S* __restrict__ w,
                                                         float* __restrict__ logits, int T, int D, int E) {
  __shared__ float part[8][NT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  float acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = 0.f;
  for (int d = threadIdx.x * 8; d < D; d += blockDim.x * 8) {
    typedef S V __attribute__((ext_vector_type(8)));
    const V wv = *reinterpret_cast<const V*>(w + (size_t)blockIdx.x * D + d);
    V xv[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)   // rows behind the last read it again
      xv[t] = *reinterpret_cast<const V*>(x + (size_t)min(t, T - 1) * D + d);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[t] = fmaf((float)xv[t][i], (float)wv[i], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float v = wave_sum_f(acc[t]);
    if (lane == 0) part[wave][t] = v;
  }
  __syncthreads();
  if ((int)threadIdx.x < T) {
    float v = 0.f;
    for (int i = 0; i < waves; ++i) v += part[i][threadIdx.x];
    logits[(size_t)threadIdx.x * E + blockIdx.x] = v;
  }
}

// Words of 64 experts that a token's choices take.
__device__ __forceinline__ int choice_words(int E) { return (E + 63) / 64; }

// Each token's k experts, as bits of chosen[t][e / 64] (LDS), a wave a token; its
// weights (global [T, E], chosen entries) where weights is not null. PER >= words.
// Ties go to the lower expert, NaN ranks below -inf, as in moe_plan_create.
template <int PER>
__device__ __forceinline__ void route_token(const FewArgs& a, int t, uint64_t* chosen, float* weights) {
  const int lane = threadIdx.x & 63;
  float l[PER];
  uint32_t key[PER], top = 0u;
  uint64_t sel[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) l[p] = lane + 64 * p < a.E ? a.logits[(size_t)t * a.E + lane + 64 * p] : 0.f;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    key[p] = lane + 64 * p < a.E ? order_key(l[p]) + 1u : 0u;   // 0: none
    sel[p] = 0ull;
  }
  for (int j = 0; j < a.k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int p = 1; p < PER; ++p) m = max(m, key[p]);
    m = wave_max_u32(m);
    if (j == 0) top = m;
    bool open = true;   // the lowest expert among equal ones
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const uint64_t at = __ballot(key[p] == m);
      const uint64_t bit = open ? at & (0ull - at) : 0ull;
      open = open && !at;
      sel[p] |= bit;
      if ((bit >> lane) & 1ull) key[p] = 0u;
    }
  }
  if (lane == 0) {
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if (64 * p < a.E) chosen[t * choice_words(a.E) + p] = sel[p];
  }
  if (!weights) return;
  const float l0 = key_value(top - 1u);
  float ex[PER], sum = 0.f;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    ex[p] = 0.f;
    if ((sel[p] >> lane) & 1ull) {
      // exp(l - l0): the difference's rounding error is put back
      const float d = l[p] - l0, back = d + l0;
      const float err = (l[p] - back) + ((back - d) - l0);
      ex[p] = expf(d);
      if (ex[p] > 0.f && err == err) ex[p] = fmaf(ex[p], err, ex[p]);
    }
    sum += ex[p];
  }
  sum = wave_sum_f(sum);
#pragma unroll
  for (int p = 0; p < PER; ++p)
    if ((sel[p] >> lane) & 1ull) weights[(size_t)t * a.E + lane + 64 * p] = ex[p] / sum;
}

// The experts in use, in order, the shared one last: their tokens (bits, after the
// limit, which keeps an expert's first ones; T <= TOKENS) and the pairs before them. list in LDS:
// [0] their number, then [cap] experts, [cap] tokens, [cap] pairs before. A wave a word of experts.
template <int TOKENS>
__device__ __forceinline__ void list_experts(const FewArgs& a, const uint64_t* chosen, int32_t* list) {
  const int lane = threadIdx.x & 63, words = choice_words(a.E);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  if (wave >= words) return;
  int n = 0, pairs = 0;
  for (int p = 0; p <= wave; ++p) {
    uint32_t m = 0u;
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) m |= (uint32_t)((chosen[t * words + p] >> lane) & 1ull) << t;
    for (int over = __popc(m) - a.limit; over > 0; --over) m &= ~(0x80000000u >> __clz((int)m));
    const uint64_t used = __ballot(m != 0u), below = (1ull << lane) - 1ull;
    int here = 0, before = pairs;
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
      const uint64_t of = __ballot((m >> t) & 1u);
      here += __popcll(of);
      before += __popcll(of & below);
    }
    if (p == wave && m) {
      const int at = 1 + n + __popcll(used & below);
      list[at] = 64 * p + lane;
      list[at + cap] = (int32_t)m;
      list[at + 2 * cap] = before;
    }
    n += __popcll(used);
    pairs += here;
  }
  if (wave == words - 1 && lane == 0) {
    if (a.n_shared) {
      list[1 + n] = a.E;
      list[1 + n + cap] = (int32_t)((1u << a.T) - 1u);
      list[1 + n + 2 * cap] = pairs;
    }
    list[0] = n + a.n_shared;
  }
}

// h, the SwiGLU's f32 output, as the second launch's matrix operand: 16-bit parts, each
// the rounding of what the ones before leave (few_hold).
template <int PARTS> struct FewH;
template <> struct FewH<2> { using T = _Float16; };
template <> struct FewH<3> { using T = __bf16; };

// v's parts at h[at], h[at + F], ..: an infinity or a NaN in the first one
__device__ __forceinline__ void split_store(void* h, int parts, size_t at, int F, float v) {
  if (parts == 3) {
    __bf16* p = (__bf16*)h + at;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const __bf16 part = (__bf16)v;
      p[(size_t)i * F] = part;
      v -= (float)part;
      if (!__builtin_isfinite(v)) v = 0.f;
    }
  } else {
    _Float16* p = (_Float16*)h + at;
    const _Float16 part = (_Float16)v;
    p[0] = part;
    v = (v - (float)part) * kRestUp;
    p[F] = (_Float16)(__builtin_isfinite(v) ? v : 0.f);
  }
}

// Both matrices' sums of waves that share strips lie in LDS at once, up to 8 tokens.
template <int NI> constexpr int kParts = NI <= 2 ? 2 : 1;

template <class S, int FMT, int NI>
__global__ __launch_bounds__(64 * kRowWaves) void few_gateup_kernel(FewArgs a, int KL) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int kPart = kRowWaves * NI * 64;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  float* part = (float*)(lds + x_lds_bytes<FMT>(a.T, KL));   // [kParts][waves][NI][64]
  uint64_t* chosen = (uint64_t*)(part + kParts<NI> * kPart);   // [kFewT][words]
  int32_t* list = (int32_t*)(chosen + kFewT * choice_words(a.E));   // [1 + 3 cap]
  const S* x = (const S*)a.x;
  const int blocks = a.D / 128, per = KL / 128;
  if (wave < a.T) {
    float* weights = blockIdx.x == 0 ? a.w : nullptr;
    if (a.E <= 128) route_token<2>(a, wave, chosen, weights);
    else if (a.E <= 256) route_token<4>(a, wave, chosen, weights);
    else route_token<16>(a, wave, chosen, weights);
  } else if (wave < 4 * NI && lane < choice_words(a.E)) {
    chosen[wave * choice_words(a.E) + lane] = 0ull;   // no token
  }
  __syncthreads();
  list_experts<4 * NI>(a, chosen, list);
  __syncthreads();
  const int n_slots = __builtin_amdgcn_readfirstlane(list[0]);
  if (blockIdx.x == 0)   // for the second launch
    for (int i = threadIdx.x; i < 1 + 3 * cap; i += blockDim.x) a.list[i] = list[i];
  const int strips = a.F / 16, items = n_slots * strips;
  const int split = wave_split(items, blocks, gridDim.x), share = 1 << split;
  const int mine = wave >> split, q = wave & (share - 1), at_once = kRowWaves >> split;
  const int rounds = (items + gridDim.x * at_once - 1) / (gridDim.x * at_once);
  for (int r = 0; r < rounds; ++r) {
    const int item = (r * at_once + mine) * gridDim.x + blockIdx.x;
    const bool any = item < items;
    const int slot = any ? item / strips : 0, f0 = any ? (item - slot * strips) * 16 : 0;
    const int expert = __builtin_amdgcn_readfirstlane(list[1 + slot]);
    const int64_t n0 = (int64_t)expert * a.F + f0;
    floatx4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const WStrip<FMT> m[2] = {weight_strip<FMT, kWhole>(a.wg, a.wgs, n0 + 16, n0, a.D),
                              weight_strip<FMT, kWhole>(a.wu, a.wus, n0 + 16, n0, a.D)};
    for (int b0 = 0; b0 < blocks; b0 += per) {
      const int n = min(per, blocks - b0);
      const int first = b0 + n * q / share, end = any ? b0 + n * (q + 1) / share : first;
      Stream<S, FMT, NI, 2, kWhole> st;
      st.start(m, first, end, a.D);
      if (r == 0 || per < blocks) {
        if (r || b0) __syncthreads();   // all waves are done with the turn before
        stage_x<S, FMT>(lds, x, a.T, b0 * 128, KL, a.D);
        __syncthreads();
      }
      st.run(m, lds, a.T, KL, b0, first, end, a.D, acc);
    }
    if (split) {
#pragma unroll
      for (int j = 0; j < 2; j += kParts<NI>) {
        if (r || j) __syncthreads();   // what was there has been read
#pragma unroll
        for (int i = 0; i < kParts<NI>; ++i)
#pragma unroll
          for (int e = 0; e < NI; ++e) part[i * kPart + (wave * NI + e) * 64 + lane] = acc[j + i][e];
        __syncthreads();
        if (q == 0) {
#pragma unroll
          for (int i = 0; i < kParts<NI>; ++i) add_shared<NI>(part + i * kPart, wave, share, acc[j + i]);
        }
      }
    }
    if (any && q == 0) {
      const uint32_t tokens = (uint32_t)list[1 + cap + slot];
      const int pair0 = list[1 + 2 * cap + slot];
      // beside 4-bit weights h lies in the codes' order within each eight values
      const int f = lane & 15, at = FMT < 0 ? f : (f & 8) | ((f & 3) << 1) | ((f >> 2) & 1);
#pragma unroll
      for (int e = 0; e < NI; ++e) {
        const int t = 4 * e + (lane >> 4);
        if ((tokens >> t) & 1u)   // a token's bit: t < T
          split_store(a.h, a.parts, (size_t)(pair0 + __popc(tokens & ((1u << t) - 1u))) * a.parts * a.F + f0 + at,
                      a.F, swiglu(acc[0][e], acc[1][e], a.clamp) * a.up);
      }
    }
  }
}

// What a wave of the second launch takes at once: R = 16 output columns of kW blocks of
// 128 of an expert's F (4-bit: two, a cache line of each row; else one), or R = 8
// columns of two blocks, the first's weight rows as rows 0 .. 7 of a strip, the second's
// as rows 8 .. 15; each of the kN blocks' h is then multiplied by all 16, and the half
// of the products that belongs to the other block goes nowhere.
template <int FMT, int R> struct FewUnit {
  static constexpr int kW = R == 8 || FMT < 0 ? 1 : 2;
  static constexpr int kN = R == 8 || FMT >= 0 ? 2 : 1;
  WBlock<FMT> w[kW];
};
// Units in flight a wave. Two: with four, the longer code and the whole rings of a turn
// cost more than they bring (one token on 8 of 256 4-bit experts of 4096 x 2048: 16.7
// against 14.2 us; sixteen on 16-bit ones of 2048 x 768: 55.2 against 55.6).
constexpr int kDownDepth = 2;

constexpr int kDownWaves = 16;
static_assert(kRowWaves >= kFewT, "a wave a token");

// h in LDS: a row a pair and part (parts * pair + part), KL values, then 16 bytes, whose
// first four are the pair's routing weight, over the part's power of two; behind the rows
// 256 bytes of zeros.
constexpr size_t h_row(int KL) { return (size_t)KL * 2 + 16; }

// A turn: a range of F and the experts s0 .. s1 - 1, as many as LDS holds h of; its
// units go to the waves in runs, u .. last - 1.
struct DownTurn {
  int c0, nb;          // first block of the range of F, blocks
  int s0, s1, pair0;   // experts, pairs before the first
  int per, u, last;    // units an expert
  uint32_t inv;        // 2^32 / per, rounded up: fewer than 2^32 / per units
  __device__ __forceinline__ int expert_of(int unit) const { return per == 1 ? unit : (int)__umulhi(unit, inv); }
};

// h in PARTS parts, kSlots rows of a matrix operand a token: an instruction a step holds
// all parts of kGroup tokens, 4 of three parts or 8 of two. There are G such groups, each
// with sums of its own; an expert takes those that hold a token of its own (with 16 tokens
// mostly one).
template <int PARTS, class O, int FMT, int NI, int R, int G>
__global__ __launch_bounds__(64 * kDownWaves) void few_down_kernel(FewArgs a, int KL, int rows) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using S = typename FewH<PARTS>::T;
  using V = typename R16<S>::V;
  using U = FewUnit<FMT, R>;
  constexpr int kN = U::kN, kW = U::kW, kDepth = kDownDepth;
  constexpr int kSlots = PARTS == 3 ? 4 : 2, kGroup = 16 / kSlots;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  const int row = (int)h_row(KL), zeros = rows * PARTS * row;
  int* experts = (int*)(lds + zeros + 256);   // [cap]
  uint32_t* masks = (uint32_t*)(experts + cap);   // [cap]
  int* before = (int*)(masks + cap);              // [cap]
  const int n_slots = __builtin_amdgcn_readfirstlane(a.list[0]);
  for (int i = threadIdx.x; i < 3 * cap; i += blockDim.x)   // those from n_slots on are not used
    experts[i] = a.list[1 + i];
  if (threadIdx.x < 64) reinterpret_cast<uint32_t*>(lds + zeros)[threadIdx.x] = 0u;
  __syncthreads();
  const int blocks = a.F / 128, per_turn = KL / 128, d0 = blockIdx.x * R;
  const uint32_t rb = FMT < 0 ? (uint32_t)a.F * 2 : (uint32_t)a.F / 2;
  // R = 8: whether this lane's weights (parameters, products) are the second block's
  const bool second = FMT < 0 ? (lane & 15) >= 8 : lane >= 32, second_col = (lane & 15) >= 8;

  // the next turn, false after the last
  auto turn = [&](DownTurn& w) __attribute__((always_inline)) {
    w.s0 = w.s1;
    if (w.s0 >= n_slots) {
      w.s0 = 0;
      w.c0 += w.nb;
    }
    w.u = w.last = 0;
    if (w.c0 >= blocks || n_slots == 0) return false;
    w.nb = min(per_turn, blocks - w.c0);
    w.per = (w.nb + kN - 1) / kN;
    w.inv = 0xFFFFFFFFu / (uint32_t)w.per + 1u;
    w.pair0 = __builtin_amdgcn_readfirstlane(before[w.s0]);
    // one expert's rows always fit
    for (w.s1 = w.s0;;) {
      const int s = w.s1 + lane;
      const bool fits = s < n_slots && before[s] + __popc(masks[s]) - w.pair0 <= rows;
      const uint64_t no = ~__ballot(fits);
      w.s1 += no ? __builtin_ctzll(no) : 64;
      if (no) break;
    }
    const int units = (w.s1 - w.s0) * w.per;
    w.u = units * wave / kDownWaves;
    w.last = units * (wave + 1) / kDownWaves;
    return true;
  };
  // h of the turn's pairs, and their weights
  auto stage = [&](const DownTurn& w) __attribute__((always_inline)) {
    constexpr int kAhead = 4;
    const int end = __builtin_amdgcn_readfirstlane(before[w.s1 - 1] + __popc(masks[w.s1 - 1]));
    for (int i = threadIdx.x; i < (w.s1 - w.s0) * 16; i += 64 * kDownWaves) {
      const int s = w.s0 + (i >> 4), t = i & 15;
      const uint32_t m = masks[s];
      if ((m >> t) & 1u) {
        const int e = experts[s], p = before[s] - w.pair0 + __popc(m & ((1u << t) - 1u));
        float v = (e < a.E ? a.w[(size_t)t * a.E + e] : 1.f) * a.down;
        *reinterpret_cast<float*>(lds + PARTS * p * row + KL * 2) = v;
        if constexpr (PARTS == 2) *reinterpret_cast<float*>(lds + (PARTS * p + 1) * row + KL * 2) = v * (1.f / kRestUp);
      }
    }
    // sixteen lanes a row's block
    const int n = (end - w.pair0) * PARTS * w.nb, c = lane & 15;
    const auto h = make_rsrc((const S*)a.h + (size_t)w.pair0 * PARTS * a.F,
                             (uint32_t)(end - w.pair0) * (PARTS * 2u) * a.F);
    constexpr int kStep = kDownWaves * 4;
    const int dr = kStep / w.nb, db = kStep - dr * w.nb, i0 = threadIdx.x >> 4;
    int r = i0 / w.nb, b = i0 - r * w.nb;
    for (int i = i0; i < n; i += kStep * kAhead) {
      uint4 v[kAhead];
      int to[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        to[j] = r * row + b * 256 + c * 16;
        v[j] = buffer16(h, i + j * kStep < n ? (uint32_t)(r * a.F + (w.c0 + b) * 128 + c * 8) * 2u : kPastEnd, 0);
        r += dr;
        b += db;
        if (b >= w.nb) { b -= w.nb; ++r; }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j * kStep < n) *reinterpret_cast<uint4*>(lds + to[j]) = v[j];
    }
  };
  // unit u's weights; none from the run's end on
  auto load = [&](U& n, const DownTurn& w, int u) __attribute__((always_inline)) {
    const bool any = u < w.last;
    const int slot = any ? w.s0 + w.expert_of(u) : 0;
    const int kb = any ? w.c0 + (u - (slot - w.s0) * w.per) * kN : 0, end = any ? w.c0 + w.nb : 0;
    const int expert = __builtin_amdgcn_readfirstlane(experts[slot]);
    const int64_t n0 = (int64_t)expert * a.D + d0;
    WStrip<FMT> m = weight_strip<FMT, kWhole>(a.wd, a.wds, n0 + R, n0, a.F);
    if constexpr (R == 8) {
      const bool odd = kb + 1 >= end;   // no second block
      if (second) m.vq = odd ? kPastEnd : m.vq - 8u * rb + (FMT < 0 ? 256u : 64u);
      if constexpr (FMT >= 0) {
        using Q = Q4F<FMT>;
        if (second_col && lane < 16)
          m.vp = odd ? kPastEnd : m.vp - 8u * ((uint32_t)(a.F / Q::kGroup) * Q::kPB) + 128 / Q::kGroup * Q::kPB;
      }
    }
    constexpr bool kPair = kW == 2 && FMT != 1;   // parameters of both blocks: 16 bytes a row
#pragma unroll
    for (int j = 0; j < kW; ++j) n.w[j] = load_wblock<FMT, kWhole, !kPair>(m, kb + j, end, a.F);
    if constexpr (kPair) {
      using Q = Q4F<FMT>;
      const uint4 p = buffer16(m.p, kb < end ? run_at(m.vp, kb, 128 / Q::kGroup * Q::kPB) : kNoLoad);
      n.w[0].p[0] = p.x; n.w[0].p[1] = p.y;
      n.w[kW - 1].p[0] = p.z; n.w[kW - 1].p[1] = p.w;
    }
  };

  // what the lane reads of h, a token's part; what it adds to, the token of element e (both
  // within a group)
  const int my_token = fragment_token() / kSlots, my_part = fragment_token() % kSlots;
  auto token = [&](int e) { return kSlots == 4 ? e : 2 * e + (lane >> 5); };
  // the second of two parts has a weight of its own
  const int weight_at = KL * 2 + (PARTS == 2 && (lane & 16) ? row : 0);
  float sum[G][NI];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int e = 0; e < NI; ++e) sum[g][e] = 0.f;
  auto add = [&](const U& now, const DownTurn& w, int u) __attribute__((always_inline)) {
    const int slot = w.s0 + w.expert_of(u), kb = (u - (slot - w.s0) * w.per) * kN;   // of the turn
    const uint32_t chosen = __builtin_amdgcn_readfirstlane(masks[slot]);
    const int pair = __builtin_amdgcn_readfirstlane(before[slot]) - w.pair0;
    auto row_of = [&](int t) { return PARTS * (pair + __popc(chosen & ((1u << t) - 1u))) * row; };
#pragma unroll
    for (int b = 0; b < kW; ++b) {
      if (b && kb + b >= w.nb) break;
      Q4Steps<FMT> q;
      if constexpr (FMT >= 0) {
        uint32_t prm[FMT == 1 ? 4 : 2];
        block_params<FMT, kWhole>(now.w[b], prm);
        q = q4_steps<FMT, kWhole>(now.w[b].q, prm, 4);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (G > 1 && !((chosen >> (kGroup * g)) & ((1u << kGroup) - 1u))) continue;
        // R = 8: the strip against two blocks' h
        constexpr int kH = R == 8 ? 2 : 1;
        // a lane whose token did not choose the expert reads zeros, as one behind the parts
        // does, and all do of a second block behind the last one
        const int t = kGroup * g + my_token;
        const bool in = ((chosen >> t) & 1u) && my_part < PARTS;
        const int mine = row_of(t) + my_part * row + (kb + b) * 256;
        int at[kH];
#pragma unroll
        for (int j = 0; j < kH; ++j)
          at[j] = (in && kb + b + j < w.nb ? mine + j * 256 : zeros) + (lane >> 4) * 16;
        auto h = [&](int j, int i) { return as_v8<V>(*reinterpret_cast<const uint4*>(lds + at[j] + i * 64)); };
        floatx4 acc = {0.f, 0.f, 0.f, 0.f};
        if constexpr (FMT < 0) {
          floatx4 p[kH];
#pragma unroll
          for (int j = 0; j < kH; ++j) {
            p[j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) p[j] = mfma16(h(j, i), as_v8<V>(now.w[0].q[i]), p[j]);
          }
#pragma unroll
          for (int e = 0; e < NI; ++e) acc[e] = R == 8 && second_col ? p[kH - 1][e] : p[0][e];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const V wv = q4_widen<S, FMT>(q.word[i]);
#pragma unroll
            for (int j = 0; j < kH; ++j) {
              const V v = h(j, i);
              const floatx4 c = x_constant<S, FMT>(v, floatx4{0.f, 0.f, 0.f, 0.f}), m = mfma16(v, wv, c);
              // the other block's products with a scale of zero (an infinity or a NaN of h
              // makes NaN of its token's row anyway)
              const bool own = R == 16 || second_col == (j == 1);
              const float scale = own ? q.scale(i) : 0.f;
#pragma unroll
              for (int e = 0; e < NI; ++e) acc[e] = fmaf(scale, m[e], acc[e]);
              if constexpr (FMT != 0) {
                const float bias = own ? q.bias(i) * (-1.f / kQ4Off<S, FMT>) : 0.f;
#pragma unroll
                for (int e = 0; e < NI; ++e) acc[e] = fmaf(bias, c[e], acc[e]);
              }
            }
          }
          // Here the sums end, or they sink into the branches below and every matrix
          // instruction's result with them: spills with biases and two blocks (sixteen
          // tokens of a 2048 x 768 layer 59 us, 46 so), elsewhere a looser order (142, 157 so).
          if constexpr (FMT > 0 && R == 8)
#pragma unroll
            for (int e = 0; e < NI; ++e) asm volatile("" : "+v"(acc[e]));
        }
        // a token of another expert takes nothing: its zeros times an infinite weight are NaN
#pragma unroll
        for (int e = 0; e < NI; ++e) {
          const int to = kGroup * g + token(e);
          if ((chosen >> to) & 1u)
            sum[g][e] = fmaf(*reinterpret_cast<const float*>(lds + row_of(to) + weight_at), acc[e], sum[g][e]);
        }
      }
    }
  };

  DownTurn now{0, 0, 0, 0, 0, 0, 0, 0, 0};
  bool open = turn(now);
  U ring[kDepth];
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load(ring[i], now, now.u + i);
  while (open) {
    stage(now);
    __syncthreads();
    DownTurn next = now;
    open = turn(next);
    // in whole rings: the last one's places are filled for the next turn
    do {
      const bool end = now.u + kDepth >= now.last;
      const DownTurn from = end ? next : now;
      const int u = end ? next.u : now.u + kDepth;
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        if (now.u + i < now.last) add(ring[i], now, now.u + i);
        load(ring[i], from, u + i);
      }
      now.u += kDepth;
    } while (now.u < now.last);
    now = next;
    __syncthreads();   // all waves are done with the turn
  }
  constexpr int kSums = G * NI;
  float* part = (float*)lds;   // [waves][kSums][64]
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int e = 0; e < NI; ++e) part[(wave * kSums + g * NI + e) * 64 + lane] = sum[g][e];
  __syncthreads();
  if (threadIdx.x < 64 * kSums) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) v += part[w * kSums * 64 + threadIdx.x];
    if constexpr (R == 8) v += __shfl_xor(v, 8);   // the two blocks
    v += __shfl_xor(v, 16);                         // the parts
    if constexpr (kSlots == 4) v += __shfl_xor(v, 32);
    const int t = kGroup * (wave / NI) + token(wave % NI), c = lane & 15;
    if (t < a.T && c < R && (lane & (16 * (kSlots - 1))) == 0)
      static_cast<O*>(a.y)[(size_t)t * a.D + d0 + c] = (O)v;
  }
}

template <class S, int FMT>
hipError_t gateup_launch(const FewArgs& a, int ncu, hipStream_t s) {
  const int ni = a.T <= 4 ? 1 : a.T <= 8 ? 2 : 4;
  const size_t other = (size_t)kRowWaves * (ni <= 2 ? 2 : 1) * ni * 256 + (size_t)8 * kFewT * ((a.E + 63) / 64)
                     + (size_t)4 * (1 + 3 * few_slots(a.T, a.E, a.k, a.n_shared));
  const int KL = lds_turn(x_lds_bytes<FMT>(a.T, 128), x_lds_bytes<FMT>(a.T, 256), other, a.D);
  const size_t lds = x_lds_bytes<FMT>(a.T, KL) + other;
#define MOE_FEW(NI) \
  hipLaunchKernelGGL((few_gateup_kernel<S, FMT, NI>), dim3(ncu), dim3(64 * kRowWaves), lds, s, a, KL)
  if (ni == 1) MOE_FEW(1); else if (ni == 2) MOE_FEW(2); else MOE_FEW(4);
#undef MOE_FEW
  return hipGetLastError();
}

template <int P, class O, int FMT>
hipError_t down_launch(const FewArgs& a, int ncu, hipStream_t s) {
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  // the range of F whose rows of T tokens fit (in whole pairs of blocks, if not all of
  // it), and as many pairs' rows as there can be or fit
  const size_t other = 256 + (size_t)12 * cap, room = kLdsBytes - other;
  int KL = a.F;
  if (a.T * P * h_row(KL) > room) KL = (int)((room / (a.T * P) - 16) / 512) * 256;
  const int64_t pairs = (int64_t)a.T * (a.k + a.n_shared), fit = (int64_t)(room / (P * h_row(KL)));
  const int rows = (int)(pairs < fit ? pairs : fit);
  size_t lds = rows * P * h_row(KL) + other;
  const size_t part = (size_t)kDownWaves * 16 * 256;   // the most sums
  if (lds < part) lds = part;
#define MOE_FEW(NI, G) \
  do { \
    if (a.D / 16 >= ncu) \
      hipLaunchKernelGGL((few_down_kernel<P, O, FMT, NI, 16, G>), dim3(a.D / 16), dim3(64 * kDownWaves), lds, s, \
                         a, KL, rows); \
    else \
      hipLaunchKernelGGL((few_down_kernel<P, O, FMT, NI, 8, G>), dim3(a.D / 8), dim3(64 * kDownWaves), lds, s, \
                         a, KL, rows); \
  } while (0)
  if constexpr (P == 2) {
    if (a.T <= 2) MOE_FEW(1, 1); else if (a.T <= 4) MOE_FEW(2, 1); else if (a.T <= 8) MOE_FEW(4, 1);
    else MOE_FEW(4, 2);
  } else if constexpr (FMT < 0) {
    if (a.T == 1) MOE_FEW(1, 1); else if (a.T == 2) MOE_FEW(2, 1); else if (a.T <= 4) MOE_FEW(4, 1);
    else if (a.T <= 8) MOE_FEW(4, 2); else MOE_FEW(4, 4);
  } else {   // 4-bit layers without a limit
    if (a.T <= 4) MOE_FEW(4, 1); else MOE_FEW(4, 4);
  }
#undef MOE_FEW
  return hipGetLastError();
}

template <class S>
hipError_t gateup_fmt(const FewArgs& a, int ncu, hipStream_t s) {
  switch (a.fmt) {
    case -1: return gateup_launch<S, -1>(a, ncu, s);
    case 0: return gateup_launch<S, 0>(a, ncu, s);
    case 1: return gateup_launch<S, 1>(a, ncu, s);
    case 2: return gateup_launch<S, 2>(a, ncu, s);
    default: return hipErrorInvalidValue;
  }
}

template <int P, class O>
hipError_t down_fmt(const FewArgs& a, int ncu, hipStream_t s) {
  switch (a.fmt) {
    case 0: return down_launch<P, O, 0>(a, ncu, s);
    case 1: return down_launch<P, O, 1>(a, ncu, s);
    case 2: return down_launch<P, O, 2>(a, ncu, s);
    default: return hipErrorInvalidValue;
  }
}

template <class O>
hipError_t down_parts(const FewArgs& a, int ncu, hipStream_t s) {
  return a.parts == 3 ? down_fmt<3, O>(a, ncu, s) : down_fmt<2, O>(a, ncu, s);
}

template <class S>
hipError_t router_launch(const void* x, const void* w, float* logits, int T, int D, int E, hipStream_t s) {
  const int threads = D >= 4096 ? 512 : (D / 8 + 63) / 64 * 64;
#define MOE_FEW(NT) \
  hipLaunchKernelGGL((few_router_kernel<S, NT>), dim3(E), dim3(threads), 0, s, (const S*)x, (const S*)w, logits, \
                     T, D, E)
  if (T == 1) MOE_FEW(1); else if (T <= 4) MOE_FEW(4); else if (T <= 8) MOE_FEW(8); else MOE_FEW(16);
#undef MOE_FEW
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few_router(const void* x, int xdt, const void* w, float* logits, int T, int D, int E,
                             hipStream_t s) {
  if (xdt == MOE_BF16) return router_launch<__bf16>(x, w, logits, T, D, E, s);
  if (xdt == MOE_F16) return router_launch<_Float16>(x, w, logits, T, D, E, s);
  return hipErrorInvalidValue;
}

hipError_t launch_few_gateup(const FewArgs& a, int ncu, hipStream_t s) {
  if (a.xdt == MOE_BF16) return gateup_fmt<__bf16>(a, ncu, s);
  if (a.xdt == MOE_F16) return gateup_fmt<_Float16>(a, ncu, s);
  return hipErrorInvalidValue;
}

hipError_t launch_few_down(const FewArgs& a, int ncu, hipStream_t s) {
  const bool bf = a.xdt == MOE_BF16, f32 = a.ydt == MOE_F32;
  if (a.fmt >= 0)
    return f32 ? down_parts<float>(a, ncu, s) : bf ? down_parts<__bf16>(a, ncu, s) : down_parts<_Float16>(a, ncu, s);
  if (bf) return f32 ? down_launch<3, float, -1>(a, ncu, s) : down_launch<3, __bf16, -1>(a, ncu, s);
  return f32 ? down_launch<2, float, -1>(a, ncu, s) : down_launch<2, _Float16, -1>(a, ncu, s);
}

}  // namespace moe
