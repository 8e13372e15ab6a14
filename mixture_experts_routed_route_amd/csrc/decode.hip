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

template <class S, int FMT, int NI, int NB>
__global__ __launch_bounds__(1024) void few_gateup_kernel(FewArgs a) {
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  float* part = lds;                                   // [2][waves][2][NI][64]
  uint32_t* mask = (uint32_t*)(part + (size_t)4 * waves * NI * 64);   // [E]
  int* experts = (int*)(mask + a.E);                   // [cap]
  uint32_t* masks = (uint32_t*)(experts + cap);        // [cap]
  int* count = (int*)(masks + cap);
  const int tok = (lane & 3) * 4 + ((lane >> 2) & 3);
  const int blocks = a.D / 128, turns = (blocks + waves * NB - 1) / (waves * NB);
  const S* xr = (const S*)a.x + (size_t)(tok < a.T ? tok : 0) * a.D;
  XBlock<S, FMT> xb[NB];
  auto load_x = [&](int turn) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int kb = (turn * NB + i) * waves + wave;
      if (kb < blocks)
        xb[i] = make_xblock<S, FMT>([&](int step) {
          const int k = kb * 128 + step * 32 + (lane >> 4) * 8;
          return tok < a.T ? ldg16(xr + k) : uint4{0u, 0u, 0u, 0u};
        });
    }
  };
  load_x(0);
  const int n_slots = route_all(a, mask, experts, masks, count);
  const int strips = a.F / 16, items = n_slots * strips;
  int half = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int slot = item / strips, f0 = (item - slot * strips) * 16;
    const size_t n = (size_t)experts[slot] * a.F + f0 + (lane & 15);
    const WRow rg = weight_row<FMT>(a.wg, a.wgs, n, a.D), ru = weight_row<FMT>(a.wu, a.wus, n, a.D);
    floatx4 g = {0.f, 0.f, 0.f, 0.f}, u = g;
    for (int turn = 0; turn < turns; ++turn) {
      WBlock<FMT> bg[NB], bu[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int kb = (turn * NB + i) * waves + wave;
        if (kb < blocks) {
          bg[i] = load_wblock<FMT, false>(rg, kb, 0);
          bu[i] = load_wblock<FMT, false>(ru, kb, 0);
        }
      }
      if (turns > 1) load_x(turn);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if ((turn * NB + i) * waves + wave < blocks) {
          block_product<S, FMT, NI>(xb[i], bg[i], g);
          block_product<S, FMT, NI>(xb[i], bu[i], u);
        }
    }
    float* p = part + half * (2 * waves * NI * 64);
    half ^= 1;
#pragma unroll
    for (int e = 0; e < NI; ++e) {
      p[((wave * 2) * NI + e) * 64 + lane] = g[e];
      p[((wave * 2 + 1) * NI + e) * 64 + lane] = u[e];
    }
    __syncthreads();
    if (threadIdx.x < 64 * NI) {
      float sg = 0.f, su = 0.f;
      for (int w = 0; w < waves; ++w) {
        sg += p[(w * 2) * NI * 64 + threadIdx.x];
        su += p[(w * 2 + 1) * NI * 64 + threadIdx.x];
      }
      const int t = 4 * wave + (lane >> 4);
      if ((masks[slot] >> t) & 1u)   // a token's bit: t < T
        split_store((S*)a.h, (S*)a.h_lo, ((size_t)slot * a.T + t) * a.F + f0 + (lane & 15),
                    swiglu(sg, su, a.clamp));
    }
  }
}

template <class S, class O, int FMT, int NI>
__global__ __launch_bounds__(1024) void few_down_kernel(FewArgs a) {
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  float* part = lds;                                   // [waves][NI][64]
  int* experts = (int*)(part + (size_t)waves * NI * 64);   // [cap]
  uint32_t* masks = (uint32_t*)(experts + cap);        // [cap]
  const int n_slots = a.slots[0];
  for (int i = threadIdx.x; i < n_slots; i += blockDim.x) {
    experts[i] = a.slots[1 + i];
    masks[i] = (uint32_t)a.slots[1 + cap + i];
  }
  __syncthreads();
  const int tok = (lane & 3) * 4 + ((lane >> 2) & 3);
  const int blocks = a.F / 128, units = n_slots * blocks;
  const int d0 = blockIdx.x * 16;
  float sum[NI];
#pragma unroll
  for (int e = 0; e < NI; ++e) sum[e] = 0.f;
  using V = typename R16<S>::V;
  for (int unit = wave; unit < units; unit += waves) {
    const int slot = unit / blocks, kb = unit - slot * blocks;
    const int expert = experts[slot];
    const uint32_t m = masks[slot];
    const WRow row = weight_row<FMT>(a.wd, a.wds, (size_t)expert * a.D + d0 + (lane & 15), a.F);
    const WBlock<FMT> wb = load_wblock<FMT, false>(row, kb, 0);
    const bool mine = (m >> tok) & 1u;
    const size_t at = ((size_t)slot * a.T + (mine ? tok : 0)) * a.F + kb * 128 + (lane >> 4) * 8;
    uint4 hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = mine ? ldg16((const S*)a.h + at + 32 * i) : uint4{0u, 0u, 0u, 0u};
      lo[i] = mine ? ldg16((const S*)a.h_lo + at + 32 * i) : uint4{0u, 0u, 0u, 0u};
    }
    float wt[NI];
    bool in[NI];
#pragma unroll
    for (int e = 0; e < NI; ++e) {
      const int t = 4 * e + (lane >> 4);
      in[e] = (m >> t) & 1u;
      wt[e] = in[e] && expert < a.E ? a.w[(size_t)t * a.E + expert] : 1.f;
    }
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
    const XBlock<S, FMT> xh = make_xblock<S, FMT>([&](int i) { return hi[i]; });
    const XBlock<S, FMT> xl = make_xblock<S, FMT>([&](int i) { return lo[i]; });
    block_product<S, FMT, NI>(xl, wb, acc);
    block_product<S, FMT, NI>(xh, wb, acc);
    // a token of another expert takes nothing: its zeros times an infinite weight are NaN
#pragma unroll
    for (int e = 0; e < NI; ++e) sum[e] = in[e] ? fmaf(wt[e], acc[e], sum[e]) : sum[e];
  }
#pragma unroll
  for (int e = 0; e < NI; ++e) part[(wave * NI + e) * 64 + lane] = sum[e];
  __syncthreads();
  if (threadIdx.x < 64 * NI) {
    float v = 0.f;
    for (int w = 0; w < waves; ++w) v += part[w * NI * 64 + threadIdx.x];
    const int t = 4 * wave + (lane >> 4);
    if (t < a.T) static_cast<O*>(a.y)[(size_t)t * a.D + d0 + (lane & 15)] = (O)v;
  }
}

template <class S, int FMT>
hipError_t gateup_launch(const FewArgs& a, int ncu, hipStream_t s) {
  const int blocks = a.D / 128;
  const int waves = blocks <= 4 ? 4 : blocks <= 16 ? 8 : 16;
  const int ni = a.T <= 4 ? 1 : a.T <= 8 ? 2 : 4;
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  const int64_t items = (int64_t)cap * (a.F / 16);
  const int grid = (int)(items < 4 * ncu ? items : 4 * ncu);
  const size_t lds = (size_t)4 * waves * ni * 256 + (size_t)4 * (a.E + 2 * cap + 1);
#define MOE_FEW(NI, NB) \
  hipLaunchKernelGGL((few_gateup_kernel<S, FMT, NI, NB>), dim3(grid), dim3(64 * waves), lds, s, a)
  if (blocks <= waves) {
    if (ni == 1) MOE_FEW(1, 1); else if (ni == 2) MOE_FEW(2, 1); else MOE_FEW(4, 1);
  } else {
    if (ni == 1) MOE_FEW(1, 2); else if (ni == 2) MOE_FEW(2, 2); else MOE_FEW(4, 2);
  }
#undef MOE_FEW
  return hipGetLastError();
}

template <class S, class O, int FMT>
hipError_t down_launch(const FewArgs& a, hipStream_t s) {
  const int ni = a.T <= 4 ? 1 : a.T <= 8 ? 2 : 4;
  const int cap = few_slots(a.T, a.E, a.k, a.n_shared);
  const int waves = 16;
  const size_t lds = (size_t)waves * ni * 256 + (size_t)8 * cap;
#define MOE_FEW(NI) \
  hipLaunchKernelGGL((few_down_kernel<S, O, FMT, NI>), dim3(a.D / 16), dim3(64 * waves), lds, s, a)
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
