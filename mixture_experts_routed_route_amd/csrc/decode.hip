// The whole layer for 1 to 16 tokens, from router logits to y, in two launches
// on gfx950 (moe_decode): no plan, no pair list, nothing between workgroups but
// the launch boundary.
//
//  * gate/up: every workgroup routes all tokens itself (a wave a token, k rounds of
//    a wave-wide maximum; the first one writes the routing for the second launch),
//    then takes (expert, 16 features) items: the expert's 16 gate and 16 up rows
//    against all tokens' rows of x at once, which stay in registers as fragments
//    (rows16.h). A token that did not choose the expert costs no memory, only
//    lanes of a matrix instruction. h is kept in two 16-bit parts, its rounding
//    and the rest (about 16 or 22 bits): the matrix units wait for memory anyway.
//  * down: a workgroup takes 16 output columns and walks all experts that were
//    chosen, its waves taking blocks of 128 of F in turn; each block's sums are
//    scaled by the routing weights in f32 and added, the waves' sums meet in LDS,
//    y is rounded once. Sums run in a fixed order: the same bits every time.
//
// Bound by the chosen experts' weights, read once.
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

// Words of 64 experts that a token's choices take.
__device__ __forceinline__ int choice_words(int E) { return (E + 63) / 64; }

// Each token's k experts, as bits of chosen[t][e / 64] (LDS), a wave a token; its
// weights (global [T, E], chosen entries) where weights is not null. PER = words.
// Ties go to the lower expert, NaN ranks below -inf, as in moe_plan_create.
template <int PER>
__device__ __forceinline__ void route_tokens(const FewArgs& a, uint64_t* chosen, float* weights) {
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int t = wave; t < a.T; t += waves) {
    float l[PER];
    uint32_t key[PER], top = 0u;
    uint64_t sel[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int e = lane + 64 * p;
      l[p] = e < a.E ? a.logits[(size_t)t * a.E + e] : 0.f;
    }
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
    if (!weights) continue;
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
}

// Expert 64 p + lane's tokens, as bits, after the limit (its first tokens stay).
__device__ __forceinline__ uint32_t tokens_of(const FewArgs& a, const uint64_t* chosen, int p) {
  const int lane = threadIdx.x & 63, words = choice_words(a.E);
  uint32_t m = 0u;
  for (int t = 0; t < a.T; ++t) m |= (uint32_t)((chosen[t * words + p] >> lane) & 1ull) << t;
  for (int over = __popc(m) - a.limit; over > 0; --over) m &= ~(0x80000000u >> __clz((int)m));
  return m;
}

// The experts in use, in order, then the shared one: their number; and expert and
// tokens of number `slot` (or of none). Every wave for itself.
__device__ __forceinline__ int experts_in_use(const FewArgs& a, const uint64_t* chosen) {
  int n = 0;
  for (int p = 0; p < choice_words(a.E); ++p) n += __popcll(__ballot(tokens_of(a, chosen, p) != 0u));
  return n + a.n_shared;
}
__device__ __forceinline__ void expert_of(const FewArgs& a, const uint64_t* chosen, int slot, int* expert,
                                          uint32_t* tokens) {
  *expert = a.E;
  *tokens = (1u << a.T) - 1u;
  int n = 0;
  for (int p = 0; p < choice_words(a.E); ++p) {
    const uint32_t m = tokens_of(a, chosen, p);
    uint64_t used = __ballot(m != 0u);
    const int here = __popcll(used);
    if (slot < n + here) {   // wave-uniform
      for (int i = n; i < slot; ++i) used &= used - 1ull;
      const int l = __builtin_ctzll(used);
      *expert = 64 * p + l;
      *tokens = (uint32_t)__builtin_amdgcn_readlane((int)m, l);
      return;
    }
    n += here;
  }
}

// Routing of all tokens into chosen[T][words] (LDS); the first workgroup writes what
// the second launch reads: the weights, and the experts in use with their tokens.
__device__ __forceinline__ void route_all(const FewArgs& a, uint64_t* chosen) {
  float* weights = blockIdx.x == 0 ? a.w : nullptr;
  if (a.E <= 128) route_tokens<2>(a, chosen, weights);
  else if (a.E <= 256) route_tokens<4>(a, chosen, weights);
  else route_tokens<16>(a, chosen, weights);
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x < 64) {
    const int lane = threadIdx.x, cap = few_slots(a.T, a.E, a.k, a.n_shared);
    int n = 0;
    for (int p = 0; p < choice_words(a.E); ++p) {
      const uint32_t m = tokens_of(a, chosen, p);
      const uint64_t used = __ballot(m != 0u);
      if (m) {
        const int at = n + __popcll(used & ((1ull << lane) - 1ull));
        a.slots[1 + at] = 64 * p + lane;
        a.slots[1 + cap + at] = (int32_t)m;
      }
      n += __popcll(used);
    }
    if (lane == 0) {
      if (a.n_shared) {
        a.slots[1 + n] = a.E;
        a.slots[1 + cap + n] = (int32_t)((1u << a.T) - 1u);
      }
      a.slots[0] = n + a.n_shared;
    }
  }
}

// h's rounding at h[at], the rest at h[at + F].
template <class S>
__device__ __forceinline__ void split_store(S* h, size_t at, int F, float v) {
  const S hi = (S)v;
  h[at] = hi;
  // an infinity stays one: inf - inf would make the sum of the parts a NaN
  const float rest = v - (float)hi;
  h[at + F] = (S)(rest == rest ? rest : 0.f);
}

template <class S, int FMT, int NI>
__global__ __launch_bounds__(64 * kRowWaves) void few_gateup_kernel(FewArgs a, int KL) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* part = (float*)(lds + x_lds_bytes<FMT>(a.T, KL));   // [waves][NI][64]
  uint64_t* chosen = (uint64_t*)(part + kRowWaves * NI * 64);   // [T][words]
  const S* x = (const S*)a.x;
  const int blocks = a.D / 128, per = KL / 128;
  route_all(a, chosen);
  const int strips = a.F / 16, items = experts_in_use(a, chosen) * strips;
  const int split = wave_split(items, blocks, gridDim.x), share = 1 << split;
  const int mine = wave >> split, q = wave & (share - 1), at_once = kRowWaves >> split;
  const int rounds = (items + gridDim.x * at_once - 1) / (gridDim.x * at_once);
  for (int r = 0; r < rounds; ++r) {
    const int item = (r * at_once + mine) * gridDim.x + blockIdx.x;
    const bool any = item < items;
    const int slot = any ? item / strips : 0, f0 = any ? (item - slot * strips) * 16 : 0;
    int expert;
    uint32_t tokens;
    expert_of(a, chosen, slot, &expert, &tokens);
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
      for (int j = 0; j < 2; ++j) {
        if (r || j) __syncthreads();   // what was there has been read
#pragma unroll
        for (int e = 0; e < NI; ++e) part[(wave * NI + e) * 64 + lane] = acc[j][e];
        __syncthreads();
        if (q == 0) add_shared<NI>(part, wave, share, acc[j]);
      }
    }
    if (any && q == 0) {
      // beside 4-bit weights h lies in the codes' order within each eight values
      const int f = lane & 15, at = FMT < 0 ? f : (f & 8) | ((f & 3) << 1) | ((f >> 2) & 1);
#pragma unroll
      for (int e = 0; e < NI; ++e) {
        const int t = 4 * e + (lane >> 4);
        if ((tokens >> t) & 1u)   // a token's bit: t < T
          split_store((S*)a.h, ((size_t)slot * a.T + t) * 2 * a.F + f0 + at, a.F,
                      swiglu(acc[0][e], acc[1][e], a.clamp));
      }
    }
  }
}

// What a wave of the second launch takes at once: R = 16 output columns of kW blocks of
// 128 of an expert's F (4-bit: two, a cache line of each row; else one), or R = 8
// columns of two blocks, the first's weight rows as rows 0 .. 7 of a strip, the second's
// as rows 8 .. 15; each of the kN blocks' h is then multiplied by all 16, and the half
// of the products that belongs to the other block goes nowhere.
// h's two parts: up to 8 tokens have both in one fragment (PARTS 1: row 2 t of h and row
// 2 t + 1 are two of its 16), more have a fragment of each (PARTS 2).
template <int FMT, int R, int PARTS> struct FewUnit {
  static constexpr int kW = R == 8 || FMT < 0 ? 1 : 2;
  static constexpr int kN = R == 8 || FMT >= 0 ? 2 : 1;
  WBlock<FMT> w[kW];
  uint4 h[kN][PARTS][4];
};

// Waves of a workgroup: h's fragments of more than 8 tokens beside 4-bit weights take
// half of a compute unit's registers in 8.
template <int FMT, int PARTS> constexpr int kDownWaves = FMT >= 0 && PARTS == 2 ? 8 : 16;

template <class S, class O, int FMT, int NI, int R, int PARTS>
__global__ __launch_bounds__(64 * (kDownWaves<FMT, PARTS>)) void few_down_kernel(FewArgs a) {
  constexpr int kWaves = kDownWaves<FMT, PARTS>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using V = typename R16<S>::V;
  using U = FewUnit<FMT, R, PARTS>;
  constexpr int kN = U::kN, kW = U::kW;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  float* part = (float*)lds;                           // [waves][NI][64]
  int* experts = (int*)(part + kWaves * NI * 64);   // [cap]
  uint32_t* masks = (uint32_t*)(experts + cap);        // [cap]
  float* weights = (float*)(masks + cap);              // [cap, T]
  const int n_slots = __builtin_amdgcn_readfirstlane(a.slots[0]);
  for (int i = threadIdx.x; i < cap; i += blockDim.x) {   // those from n_slots on are not used
    experts[i] = a.slots[1 + i];
    masks[i] = (uint32_t)a.slots[1 + cap + i];
  }
  __syncthreads();
  const int blocks = a.F / 128, per = (blocks + kN - 1) / kN, units = n_slots * per;
  const int d0 = blockIdx.x * R;
  const uint32_t hbytes = (uint32_t)(a.T * a.F) * 4;
  const uint32_t rb = FMT < 0 ? (uint32_t)a.F * 2 : (uint32_t)a.F / 2;
  // R = 8: whether this lane's weights (parameters, products) are the second block's
  const bool second = FMT < 0 ? (lane & 15) >= 8 : lane >= 32, second_col = (lane & 15) >= 8;
  // the row of h in the lane's row of a fragment: 2 t + part, or 2 t
  const int vrow = PARTS == 1 ? fragment_token() : 2 * fragment_token();
  // units go to the waves in runs
  const int first = units * wave / kWaves, last = units * (wave + 1) / kWaves;
  auto load = [&](int u) {
    U n;
    const bool any = u < last;
    const int slot = any ? u / per : 0, kb = any ? (u - slot * per) * kN : 0;
    const int expert = __builtin_amdgcn_readfirstlane(experts[slot]);
    const uint32_t chosen = __builtin_amdgcn_readfirstlane(masks[slot]);
    const int64_t n0 = (int64_t)expert * a.D + d0;
    WStrip<FMT> m = weight_strip<FMT, kWhole>(a.wd, a.wds, n0 + R, n0, a.F);
    if constexpr (R == 8) {
      const bool odd = kb + 1 >= blocks;   // no second block
      if (second) m.vq = odd ? kPastEnd : m.vq - 8u * rb + (FMT < 0 ? 256u : 64u);
      if constexpr (FMT >= 0) {
        using Q = Q4F<FMT>;
        if (second_col && lane < 16)
          m.vp = odd ? kPastEnd : m.vp - 8u * ((uint32_t)(a.F / Q::kGroup) * Q::kPB) + 128 / Q::kGroup * Q::kPB;
      }
    }
#pragma unroll
    for (int j = 0; j < kW; ++j)
      n.w[j] = load_wblock<FMT, kWhole>(m, kb + j, any ? blocks : 0, a.F);
    const auto rh = make_rsrc((const S*)a.h + (size_t)slot * a.T * 2 * a.F, hbytes);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      // a lane whose token did not choose the expert reads zeros
      const uint32_t v = any && kb + j < blocks && ((chosen >> (vrow >> 1)) & 1u)
          ? (uint32_t)(vrow * a.F + (kb + j) * 128 + (lane >> 4) * 8) * 2 : kPastEnd;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < PARTS; ++p) n.h[j][p][i] = buffer16(rh, v + 64 * i, (uint32_t)(p * a.F) * 2);
    }
    return n;
  };
  float sum[NI];
#pragma unroll
  for (int e = 0; e < NI; ++e) sum[e] = 0.f;
  U next = load(first);
  for (int i = threadIdx.x; i < n_slots * a.T; i += blockDim.x) {
    const int slot = i / a.T, t = i - slot * a.T, e = experts[slot];
    weights[i] = e < a.E && ((masks[slot] >> t) & 1u) ? a.w[(size_t)t * a.E + e] : 1.f;
  }
  __syncthreads();
  // the token of element e
  auto token = [&](int e) { return PARTS == 1 ? 2 * e + (lane >> 5) : 4 * e + (lane >> 4); };
  for (int u = first; u < last; ++u) {
    const U now = next;
    next = load(u + 1);
    const int slot = u / per;
    const uint32_t chosen = __builtin_amdgcn_readfirstlane(masks[slot]);
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
    if constexpr (FMT < 0) {
      floatx4 p[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        p[j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int q = PARTS - 1; q >= 0; --q)
            p[j] = mfma16(as_v8<V>(now.h[j][q][i]), as_v8<V>(now.w[0].q[i]), p[j]);
      }
#pragma unroll
      for (int e = 0; e < NI; ++e) acc[e] = R == 8 && second_col ? p[kN - 1][e] : p[0][e];
    } else {
#pragma unroll
      for (int b = 0; b < kW; ++b) {
        uint32_t prm[FMT == 1 ? 4 : 2];
        block_params<FMT, kWhole>(now.w[b], prm);
        const Q4Steps<FMT> q = q4_steps<FMT, kWhole>(now.w[b].q, prm, 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const V w = q4_widen<S, FMT>(q.word[i]);
          // R = 8: the strip against both blocks' h; R = 16: a strip a block
          constexpr int kH = R == 8 ? 2 : 1;
          floatx4 m[kH], c[kH];
#pragma unroll
          for (int j = 0; j < kH; ++j) {
            c[j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = PARTS - 1; p >= 0; --p) c[j] = x_constant<S, FMT>(as_v8<V>(now.h[b + j][p][i]), c[j]);
            m[j] = c[j];
#pragma unroll
            for (int p = PARTS - 1; p >= 0; --p) m[j] = mfma16(as_v8<V>(now.h[b + j][p][i]), w, m[j]);
          }
#pragma unroll
          for (int e = 0; e < NI; ++e) {
            const bool o = R == 8 && second_col;
            acc[e] = fmaf(q.scale(i), o ? m[kH - 1][e] : m[0][e], acc[e]);
            if constexpr (FMT != 0)
              acc[e] = fmaf(q.bias(i) * (-1.f / kQ4Off<S, FMT>), o ? c[kH - 1][e] : c[0][e], acc[e]);
          }
        }
      }
    }
    // a token of another expert takes nothing: its zeros times an infinite weight are NaN
#pragma unroll
    for (int e = 0; e < NI; ++e)
      if ((chosen >> token(e)) & 1u) sum[e] = fmaf(weights[slot * a.T + token(e)], acc[e], sum[e]);
  }
#pragma unroll
  for (int e = 0; e < NI; ++e) part[(wave * NI + e) * 64 + lane] = sum[e];
  __syncthreads();
  if (threadIdx.x < 64 * NI) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w * NI * 64 + threadIdx.x];
    if constexpr (R == 8) v += __shfl_xor(v, 8);        // the two blocks
    if constexpr (PARTS == 1) v += __shfl_xor(v, 16);   // the two parts
    const int t = token(wave), c = lane & 15;
    if (t < a.T && c < R && (PARTS == 2 || !(lane & 16)))
      static_cast<O*>(a.y)[(size_t)t * a.D + d0 + c] = (O)v;
  }
}

template <class S, int FMT>
hipError_t gateup_launch(const FewArgs& a, int ncu, hipStream_t s) {
  const int ni = a.T <= 4 ? 1 : a.T <= 8 ? 2 : 4;
  const size_t other = (size_t)kRowWaves * ni * 256 + (size_t)8 * a.T * ((a.E + 63) / 64);
  const int KL = lds_turn(x_lds_bytes<FMT>(a.T, 128), x_lds_bytes<FMT>(a.T, 256), other, a.D);
  const size_t lds = x_lds_bytes<FMT>(a.T, KL) + other;
#define MOE_FEW(NI) \
  hipLaunchKernelGGL((few_gateup_kernel<S, FMT, NI>), dim3(ncu), dim3(64 * kRowWaves), lds, s, a, KL)
  if (ni == 1) MOE_FEW(1); else if (ni == 2) MOE_FEW(2); else MOE_FEW(4);
#undef MOE_FEW
  return hipGetLastError();
}

template <class S, class O, int FMT>
hipError_t down_launch(const FewArgs& a, int ncu, hipStream_t s) {
  const int ni = a.T <= 2 ? 1 : a.T <= 4 ? 2 : 4;   // with both parts of h; above 8 tokens, of one
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  const size_t lds = (size_t)kRowWaves * ni * 256 + (size_t)4 * cap * (2 + a.T);
#define MOE_FEW(NI, R, PARTS) \
  hipLaunchKernelGGL((few_down_kernel<S, O, FMT, NI, R, PARTS>), dim3(a.D / R), \
                     dim3(64 * (kDownWaves<FMT, PARTS>)), lds, s, a)
  if (a.D / 16 >= ncu) {
    if (ni == 1) MOE_FEW(1, 16, 1); else if (ni == 2) MOE_FEW(2, 16, 1);
    else if (a.T <= 8) MOE_FEW(4, 16, 1); else MOE_FEW(4, 16, 2);
  } else {
    if (ni == 1) MOE_FEW(1, 8, 1); else if (ni == 2) MOE_FEW(2, 8, 1);
    else if (a.T <= 8) MOE_FEW(4, 8, 1); else MOE_FEW(4, 8, 2);
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

template <class S, class O>
hipError_t down_fmt(const FewArgs& a, int ncu, hipStream_t s) {
  switch (a.fmt) {
    case -1: return down_launch<S, O, -1>(a, ncu, s);
    case 0: return down_launch<S, O, 0>(a, ncu, s);
    case 1: return down_launch<S, O, 1>(a, ncu, s);
    case 2: return down_launch<S, O, 2>(a, ncu, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_few_gateup(const FewArgs& a, int ncu, hipStream_t s) {
  if (a.xdt == MOE_BF16) return gateup_fmt<__bf16>(a, ncu, s);
  if (a.xdt == MOE_F16) return gateup_fmt<_Float16>(a, ncu, s);
  return hipErrorInvalidValue;
}

hipError_t launch_few_down(const FewArgs& a, int ncu, hipStream_t s) {
  if (a.xdt == MOE_BF16)
    return a.ydt == MOE_F32 ? down_fmt<__bf16, float>(a, ncu, s) : down_fmt<__bf16, __bf16>(a, ncu, s);
  if (a.xdt == MOE_F16)
    return a.ydt == MOE_F32 ? down_fmt<_Float16, float>(a, ncu, s) : down_fmt<_Float16, _Float16>(a, ncu, s);
  return hipErrorInvalidValue;
}

}  // namespace moe
