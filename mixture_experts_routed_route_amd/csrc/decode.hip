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

// The tokens that chose each expert, as bits of mask[e] (LDS, zeroed); weights
// (global [T, E], chosen entries) where weights is not null. PER logits a lane.
// Ties go to the lower expert, NaN ranks below -inf, as in moe_plan_create.
template <int PER>
__device__ __forceinline__ void route_tokens(const FewArgs& a, uint32_t* mask, float* weights) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int t = wave; t < a.T; t += waves) {
    float l[PER];
    uint32_t key[PER], sel = 0u, top = 0u;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int e = lane + 64 * p;
      l[p] = e < a.E ? a.logits[(size_t)t * a.E + e] : 0.f;
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) key[p] = lane + 64 * p < a.E ? order_key(l[p]) + 1u : 0u;   // 0: none
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
        if (open && at) {
          open = false;
          if (lane == __builtin_ctzll(at)) {
            key[p] = 0u;
            sel |= 1u << p;
          }
        }
      }
    }
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if ((sel >> p) & 1u) atomicOr(&mask[lane + 64 * p], 1u << t);
    if (!weights) continue;
    const float l0 = key_value(top - 1u);
    float ex[PER], sum = 0.f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      ex[p] = 0.f;
      if ((sel >> p) & 1u) {
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
      if ((sel >> p) & 1u) weights[(size_t)t * a.E + lane + 64 * p] = ex[p] / sum;
  }
}

// Routing of all tokens: the experts in use, in order, and their tokens' masks
// after the limit, in LDS (experts[slot], masks[slot]); returns their number.
// The first workgroup writes them and the weights for the second launch.
__device__ __forceinline__ int route_all(const FewArgs& a, uint32_t* mask, int* experts, uint32_t* masks,
                                         int* count) {
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) mask[e] = 0u;
  __syncthreads();
  float* weights = blockIdx.x == 0 ? a.w : nullptr;
  if (a.E <= 128) route_tokens<2>(a, mask, weights);
  else if (a.E <= 256) route_tokens<4>(a, mask, weights);
  else route_tokens<16>(a, mask, weights);
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int n = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      uint32_t m = e0 + lane < a.E ? mask[e0 + lane] : 0u;
      // the first `limit` tokens stay
      for (int over = __popc(m) - a.limit; over > 0; --over) m &= ~(0x80000000u >> __clz((int)m));
      const uint64_t used = __ballot(m != 0u);
      if (m) {
        const int at = n + __popcll(used & ((1ull << lane) - 1ull));
        experts[at] = e0 + lane;
        masks[at] = m;
      }
      n += __popcll(used);
    }
    if (a.n_shared) {
      if (lane == 0) {
        experts[n] = a.E;
        masks[n] = (1u << a.T) - 1u;
      }
      ++n;
    }
    if (lane == 0) *count = n;
  }
  __syncthreads();
  const int n = *count;
  if (blockIdx.x == 0) {
    const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      a.slots[1 + i] = experts[i];
      a.slots[1 + cap + i] = (int32_t)masks[i];
    }
    if (threadIdx.x == 0) a.slots[0] = n;
  }
  return n;
}

template <class S>
__device__ __forceinline__ void split_store(S* hi, S* lo, size_t at, float h) {
  const S v = (S)h;
  hi[at] = v;
  // an infinity stays one: inf - inf would make the sum of the parts a NaN
  const float rest = h - (float)v;
  lo[at] = (S)(rest == rest ? rest : 0.f);
}

template <class S, int FMT, int NI>
__global__ __launch_bounds__(64 * kRowWaves) void few_gateup_kernel(FewArgs a, int KL) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  float* part = (float*)(lds + x_lds_bytes<FMT>(a.T, KL));   // [waves][NI][64]
  uint32_t* mask = (uint32_t*)(part + kRowWaves * NI * 64);   // [E]
  int* experts = (int*)(mask + a.E);                   // [cap]
  uint32_t* masks = (uint32_t*)(experts + cap);        // [cap]
  int* count = (int*)(masks + cap);
  const S* x = (const S*)a.x;
  const int blocks = a.D / 128, per = KL / 128;
  if (per >= blocks) stage_x<S, FMT>(lds, x, a.T, 0, KL, a.D);
  const int n_slots = __builtin_amdgcn_readfirstlane(route_all(a, mask, experts, masks, count));
  const int strips = a.F / 16, items = n_slots * strips;
  const int split = wave_split(items, blocks, gridDim.x), share = 1 << split;
  const int mine = wave >> split, q = wave & (share - 1), at_once = kRowWaves >> split;
  const int rounds = (items + gridDim.x * at_once - 1) / (gridDim.x * at_once);
  for (int r = 0; r < rounds; ++r) {
    const int item = (r * at_once + mine) * gridDim.x + blockIdx.x;
    const bool any = item < items;
    const int slot = any ? item / strips : 0, f0 = any ? (item - slot * strips) * 16 : 0;
    const int expert = __builtin_amdgcn_readfirstlane(experts[slot]);
    const int64_t n0 = (int64_t)expert * a.F + f0;
    floatx4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const WStrip<FMT> m[2] = {weight_strip<FMT, kWhole>(a.wg, a.wgs, n0 + 16, n0, a.D),
                              weight_strip<FMT, kWhole>(a.wu, a.wus, n0 + 16, n0, a.D)};
    for (int b0 = 0; b0 < blocks; b0 += per) {
      const int n = min(per, blocks - b0);
      const int first = b0 + n * q / share, end = any ? b0 + n * (q + 1) / share : first;
      Stream<S, FMT, NI, 2, kWhole> st;
      st.start(m, first, end, a.D);
      if (per < blocks) {
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
        if (q == 0) {
#pragma unroll
          for (int e = 0; e < NI; ++e)
            for (int w = 1; w < share; ++w) acc[j][e] += part[((wave + w) * NI + e) * 64 + lane];
        }
      }
    }
    if (any && q == 0) {
      const uint32_t chosen = masks[slot];
#pragma unroll
      for (int e = 0; e < NI; ++e) {
        const int t = 4 * e + (lane >> 4);
        if ((chosen >> t) & 1u)   // a token's bit: t < T
          split_store((S*)a.h, (S*)a.h_lo, ((size_t)slot * a.T + t) * a.F + f0 + (lane & 15),
                      swiglu(acc[0][e], acc[1][e], a.clamp));
      }
    }
  }
}

// A block of 128 of an expert's F in the second launch: weights, both parts of h.
template <int FMT> struct FewUnit {
  WBlock<FMT> w;
  uint4 hi[4], lo[4];
};

template <class S, class O, int FMT, int NI>
__global__ __launch_bounds__(64 * kRowWaves) void few_down_kernel(FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using V = typename R16<S>::V;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  float* part = (float*)lds;                           // [waves][NI][64]
  int* experts = (int*)(part + kRowWaves * NI * 64);   // [cap]
  uint32_t* masks = (uint32_t*)(experts + cap);        // [cap]
  float* weights = (float*)(masks + cap);              // [cap, T]
  const int n_slots = __builtin_amdgcn_readfirstlane(a.slots[0]);
  for (int i = threadIdx.x; i < n_slots * a.T; i += blockDim.x) {
    const int slot = i / a.T, t = i - slot * a.T;
    const int e = a.slots[1 + slot];
    const uint32_t m = (uint32_t)a.slots[1 + cap + slot];
    weights[i] = e < a.E && ((m >> t) & 1u) ? a.w[(size_t)t * a.E + e] : 1.f;
    if (t == 0) {
      experts[slot] = e;
      masks[slot] = m;
    }
  }
  __syncthreads();
  const int tok = fragment_token();
  const int blocks = a.F / 128, units = n_slots * blocks;
  const int d0 = blockIdx.x * 16;
  const uint32_t hbytes = (uint32_t)(a.T * a.F) * 2;
  // unit u: its loads; a lane whose token did not choose the expert reads zeros
  auto load = [&](int u) {
    FewUnit<FMT> n;
    const bool any = u < units;
    const int slot = any ? u / blocks : 0, kb = any ? u - slot * blocks : 0;
    const int expert = __builtin_amdgcn_readfirstlane(experts[slot]);
    const uint32_t chosen = __builtin_amdgcn_readfirstlane(masks[slot]);
    const int64_t n0 = (int64_t)expert * a.D + d0;
    const WStrip<FMT> m = weight_strip<FMT, kWhole>(a.wd, a.wds, n0 + 16, n0, a.F);
    n.w = load_wblock<FMT, kWhole>(m, kb, any ? blocks : 0, a.F);
    const auto rh = make_rsrc((const S*)a.h + (size_t)slot * a.T * a.F, hbytes);
    const auto rl = make_rsrc((const S*)a.h_lo + (size_t)slot * a.T * a.F, hbytes);
    const uint32_t v = any && ((chosen >> tok) & 1u)
        ? (uint32_t)(tok * a.F + kb * 128 + (lane >> 4) * 8) * 2 : kPastEnd;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n.hi[i] = buffer16(rh, v + 64 * i, 0);
      n.lo[i] = buffer16(rl, v + 64 * i, 0);
    }
    return n;
  };
  float sum[NI];
#pragma unroll
  for (int e = 0; e < NI; ++e) sum[e] = 0.f;
  FewUnit<FMT> next = load(wave);
  for (int u = wave; u < units; u += kRowWaves) {
    const FewUnit<FMT> now = next;
    next = load(u + kRowWaves);
    const int slot = u / blocks;
    const uint32_t chosen = __builtin_amdgcn_readfirstlane(masks[slot]);
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
    if constexpr (FMT < 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc = mfma16(as_v8<V>(now.lo[i]), as_v8<V>(now.w.q[i]), acc);
        acc = mfma16(as_v8<V>(now.hi[i]), as_v8<V>(now.w.q[i]), acc);
      }
    } else {
      const Q4Steps<FMT> q = q4_steps<FMT, kWhole>(now.w, 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const V hi = as_v8<V>(q4_order(now.hi[i])), lo = as_v8<V>(q4_order(now.lo[i]));
        const V w = q4_widen<S, FMT>(q.word[i]);
        const floatx4 c = x_constant<S, FMT>(hi, x_constant<S, FMT>(lo, floatx4{0.f, 0.f, 0.f, 0.f}));
        const floatx4 m = mfma16(hi, w, mfma16(lo, w, c));
#pragma unroll
        for (int e = 0; e < NI; ++e) {
          acc[e] = fmaf(q.scale(i), m[e], acc[e]);
          if constexpr (FMT != 0) acc[e] = fmaf(q.bias(i) * (-1.f / kQ4Off<S, FMT>), c[e], acc[e]);
        }
      }
    }
    // a token of another expert takes nothing: its zeros times an infinite weight are NaN
#pragma unroll
    for (int e = 0; e < NI; ++e) {
      const int t = 4 * e + (lane >> 4);
      if ((chosen >> t) & 1u) sum[e] = fmaf(weights[slot * a.T + t], acc[e], sum[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < NI; ++e) part[(wave * NI + e) * 64 + lane] = sum[e];
  __syncthreads();
  if (threadIdx.x < 64 * NI) {
    float v = 0.f;
    for (int w = 0; w < kRowWaves; ++w) v += part[w * NI * 64 + threadIdx.x];
    const int t = 4 * wave + (lane >> 4);
    if (t < a.T) static_cast<O*>(a.y)[(size_t)t * a.D + d0 + (lane & 15)] = (O)v;
  }
}

template <class S, int FMT>
hipError_t gateup_launch(const FewArgs& a, int ncu, hipStream_t s) {
  const int ni = a.T <= 4 ? 1 : a.T <= 8 ? 2 : 4;
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  const size_t other = (size_t)kRowWaves * ni * 256 + (size_t)4 * (a.E + 2 * cap + 1);
  const int KL = lds_turn(x_lds_bytes<FMT>(a.T, 128), x_lds_bytes<FMT>(a.T, 256), other, a.D);
  const size_t lds = x_lds_bytes<FMT>(a.T, KL) + other;
#define MOE_FEW(NI) \
  hipLaunchKernelGGL((few_gateup_kernel<S, FMT, NI>), dim3(ncu), dim3(64 * kRowWaves), lds, s, a, KL)
  if (ni == 1) MOE_FEW(1); else if (ni == 2) MOE_FEW(2); else MOE_FEW(4);
#undef MOE_FEW
  return hipGetLastError();
}

template <class S, class O, int FMT>
hipError_t down_launch(const FewArgs& a, hipStream_t s) {
  const int ni = a.T <= 4 ? 1 : a.T <= 8 ? 2 : 4;
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  const size_t lds = (size_t)kRowWaves * ni * 256 + (size_t)4 * cap * (2 + a.T);
#define MOE_FEW(NI) \
  hipLaunchKernelGGL((few_down_kernel<S, O, FMT, NI>), dim3(a.D / 16), dim3(64 * kRowWaves), lds, s, a)
  if (ni == 1) MOE_FEW(1); else if (ni == 2) MOE_FEW(2); else MOE_FEW(4);
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
hipError_t down_fmt(const FewArgs& a, hipStream_t s) {
  switch (a.fmt) {
    case -1: return down_launch<S, O, -1>(a, s);
    case 0: return down_launch<S, O, 0>(a, s);
    case 1: return down_launch<S, O, 1>(a, s);
    case 2: return down_launch<S, O, 2>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_few_gateup(const FewArgs& a, int ncu, hipStream_t s) {
  if (a.xdt == MOE_BF16) return gateup_fmt<__bf16>(a, ncu, s);
  if (a.xdt == MOE_F16) return gateup_fmt<_Float16>(a, ncu, s);
  return hipErrorInvalidValue;
}

hipError_t launch_few_down(const FewArgs& a, hipStream_t s) {
  if (a.xdt == MOE_BF16)
    return a.ydt == MOE_F32 ? down_fmt<__bf16, float>(a, s) : down_fmt<__bf16, __bf16>(a, s);
  if (a.xdt == MOE_F16)
    return a.ydt == MOE_F32 ? down_fmt<_Float16, float>(a, s) : down_fmt<_Float16, _Float16>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace moe
