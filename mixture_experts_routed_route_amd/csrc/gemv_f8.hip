// One-token calls (T = 1) on 8-bit weights, on gfx950.
//
// A token's k choices are k distinct experts with one pair each: the call is
// the chosen experts' weight stream, and what costs is the chain of loads
// before it and the launches around it. So a workgroup finds its expert from
// the plan's choices directly (no group list), quantises the one row it needs
// itself, and the second launch sums the pairs into y: two launches.
//
//  * gate/up: a workgroup takes (pair, 16 features), four waves sharing the
//    blocks of K, four blocks of both matrices in flight each; x's row is
//    quantised into LDS meanwhile. SwiGLU output in f32.
//  * down + sum: a workgroup takes 8 columns of every pair, a wave a pair,
//    which quantises its row of h; the pairs' outputs meet in LDS and are
//    summed in f32 in slot order with the routing weights, the shared
//    expert's last, rounded once to y's type.
//
// At D 2048, F 768, 9 pairs: 9.3 us for gate/up (28 MB) and 9.2 for down (14
// MB), chains of dependent loads and cold code rather than bandwidth: with
// W_down brought into the caches during the first launch, down took 8.6, and
// the first as much longer.
//
// The products are the strips': codes widened to f16, f32 sums; a fragment's
// 16 rows are the one row, read 16 times (an LDS broadcast).
#include "f8_common.h"

namespace moe {

namespace {

constexpr int kOneU = 4;        // gate/up: blocks of K in flight a wave
constexpr int kOneDownU = 8;    // down
constexpr int kOneCols = 8;     // down: columns a workgroup
constexpr int kOneLds = 60 * 1024;

// Quantises K values of a row (type dt) into codes and scales in LDS, by
// groups of 16 lanes: group `g` of `n` takes every n-th block.
__device__ __forceinline__ void quantise_row(const void* src, int dt, size_t at, int nkb, int g,
                                             int n, char* codes, float* scales) {
  for (int b = g; b < nkb; b += n) {
    const int k = b * 128 + (threadIdx.x & 15) * 8;
    float v[8];
    raw8_to_f32(load_raw8(src, dt, at + k), dt, v);
    const F8Scale sc = f8_scale(max16(mag_max8(v)));
    *reinterpret_cast<uint2*>(codes + k) = f8_pack8(v, sc.inv);
    if ((threadIdx.x & 15) == 0) scales[b] = sc.s;
  }
}

}  // namespace

__global__ __launch_bounds__(256) void f8_one_gateup_kernel(F8OneArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];   // codes, scales
  __shared__ float part[3][2][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int K = a.D, nkb = K / 128, strips = a.F / 16;
  const int j = blockIdx.x / strips, n0 = (blockIdx.x - j * strips) * 16;
  const int e = j < a.k ? a.ids[j] : a.E;
  const int p = j < a.k ? a.tok2pair[j] : a.offsets[a.E];
  if (p < 0) return;   // a dropped pair: no row
  const size_t at = ((size_t)e * a.F + n0 + lr) * K + lq * 16;
  const size_t sat = ((size_t)e * (a.F / 128) + (n0 >> 7)) * nkb;
  // with their scales, so that none is waited for on its own
  v8i32 w[kOneU][2];
  float ws[kOneU][2];
  auto load = [&](int kb0) {
#pragma unroll
    for (int u = 0; u < kOneU; ++u) {
      const int kb = min(kb0 + 4 * u, nkb - 1);
      w[u][0] = load_codes(a.wg + at + kb * 128);
      w[u][1] = load_codes(a.wu + at + kb * 128);
      ws[u][0] = a.wgs[sat + kb];
      ws[u][1] = a.wus[sat + kb];
    }
  };
  load(wave);
  float* const xs = reinterpret_cast<float*>(lds + K);
  quantise_row(a.x, a.xdt, 0, nkb, threadIdx.x >> 4, 16, lds, xs);
  __syncthreads();
  floatx4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  for (int kb0 = wave; kb0 < nkb; kb0 += 4 * kOneU) {
    if (kb0 != wave) load(kb0);
#pragma unroll
    for (int u = 0; u < kOneU; ++u) {
      const int kb = kb0 + 4 * u;
      if (kb >= nkb) break;   // uniform in the wave
      const Codes xc = widen(load_codes(reinterpret_cast<const uint8_t*>(lds) + kb * 128 + lq * 16));
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const floatx4 b = block_product(widen(w[u][f]), xc);
        const float sc = xs[kb] * ws[u][f];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[f][q] = fmaf(b[q], sc, acc[f][q]);
      }
    }
  }
  // every column of a fragment's product is the row: lane group q's first
  // lane holds outputs 4 q .. 4 q + 3
  if (wave && lr == 0) {
#pragma unroll
    for (int f = 0; f < 2; ++f) *reinterpret_cast<floatx4*>(&part[wave - 1][f][lq * 4]) = acc[f];
  }
  __syncthreads();
  if (wave == 0 && lr == 0) {
    float v[4];
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int f = 0; f < 2; ++f) acc[f] += *reinterpret_cast<const floatx4*>(&part[s][f][lq * 4]);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = swiglu(acc[0][q], acc[1][q], a.clamp);
    *reinterpret_cast<float4*>(a.h + (size_t)p * a.F + n0 + lq * 4) = float4{v[0], v[1], v[2], v[3]};
  }
}

__global__ __launch_bounds__(1024) void f8_one_down_kernel(F8OneArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];   // a pair: codes, scales
  __shared__ float out[16][kOneCols];
  const int lane = threadIdx.x & 63;
  const int j = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // the wave's pair
  const int lr = lane & 15, lq = lane >> 4;
  const int K = a.F, nkb = K / 128, c0 = blockIdx.x * kOneCols;
  const int e = j < a.k ? a.ids[j] : a.E;
  const int p = j < a.k ? a.tok2pair[j] : a.offsets[a.E];
  const float weight = j < a.k ? a.w[j] : 1.f;
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};   // stays zero for a dropped pair
  if (p >= 0) {   // uniform in the wave; no barrier inside
    const uint8_t* wd = a.wd + ((size_t)e * a.D + c0 + (lr & (kOneCols - 1))) * K + lq * 16;
    const float* ws = a.wds + ((size_t)e * (a.D / 128) + (c0 >> 7)) * nkb;
    v8i32 w[kOneDownU];
    float sw[kOneDownU];
    auto load = [&](int kb0) {
#pragma unroll
      for (int u = 0; u < kOneDownU; ++u) {
        const int kb = min(kb0 + u, nkb - 1);
        w[u] = load_codes(wd + kb * 128);
        sw[u] = ws[kb];
      }
    };
    load(0);
    char* const codes = lds + (size_t)j * (K + nkb * 16);
    float* const hs = reinterpret_cast<float*>(codes + K);
    quantise_row(a.h, MOE_F32, (size_t)p * K, nkb, lq, 4, codes, hs);
    // written and read by this wave alone
    asm volatile("" ::: "memory");
    wait_vm_lgkm0<63>();
    for (int kb0 = 0; kb0 < nkb; kb0 += kOneDownU) {
      if (kb0) load(kb0);
#pragma unroll
      for (int u = 0; u < kOneDownU; ++u) {
        const int kb = kb0 + u;
        if (kb >= nkb) break;
        const Codes xc = widen(load_codes(reinterpret_cast<const uint8_t*>(codes) + kb * 128 + lq * 16));
        const floatx4 b = block_product(widen(w[u]), xc);
        const float sc = hs[kb] * sw[u];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = fmaf(b[q], sc, acc[q]);
      }
    }
  }
  if (lr == 0 && lq * 4 < kOneCols) {
#pragma unroll
    for (int q = 0; q < 4; ++q) out[j][lq * 4 + q] = p >= 0 ? weight * acc[q] : 0.f;
  }
  __syncthreads();
  if (threadIdx.x < kOneCols) {
    float y = 0.f;
    for (int i = 0; i < a.k + a.n_shared; ++i) y += out[i][threadIdx.x];
    store_out1(a.y, a.ydt, (size_t)c0 + threadIdx.x, y);
  }
}

static size_t one_down_lds(int F, int pairs) { return (size_t)pairs * (F + F / 128 * 16); }

bool f8_one_fits(int D, int F, int k, int n_shared) {
  return k + n_shared <= 16 && D + D / 128 * 4 <= kOneLds &&
         one_down_lds(F, k + n_shared) <= (size_t)kOneLds;
}

hipError_t launch_f8_one_gateup(const F8OneArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(f8_one_gateup_kernel, dim3((a.k + a.n_shared) * (a.F / 16)), dim3(256),
                     a.D + a.D / 128 * 4, s, a);
  return hipGetLastError();
}

hipError_t launch_f8_one_down(const F8OneArgs& a, hipStream_t s) {
  const int pairs = a.k + a.n_shared;
  hipLaunchKernelGGL(f8_one_down_kernel, dim3(a.D / kOneCols), dim3(64 * pairs),
                     one_down_lds(a.F, pairs), s, a);
  return hipGetLastError();
}

}  // namespace moe
