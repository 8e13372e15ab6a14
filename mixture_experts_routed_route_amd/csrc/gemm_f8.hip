// Products on 8-bit blocks on gfx950: e4m3 rows with a scale per row and
// 128 values times e4m3 weights with a scale per 128 x 128 block.
//
//   out[row, n] = sum_b As[row, b] Bs[n / 128, b] (sum_{k in b} A[row, k] B[n, k])
//
// The codes become f16 on the way to the matrix units, exactly (e4m3 has
// fewer exponent and fraction bits), and four v_mfma 16x16x32 sum a block of
// 128 in f32. (The 8-bit matrix instructions align each eight neighbouring
// products to the largest and drop its bits below 2^-13: 256 * 256 + 2 * 2
// sums to 65536. The 16-bit ones keep f32's 24 bits, and a strip waits for
// its weights, not for the matrix units.) The
// block's sum is scaled and added to the f32 accumulator, one fma a value.
// The weights are the matrix instruction's first operand and the rows its
// second, so a lane holds four neighbouring outputs of one row and the row's
// scale, and the weights' scale is uniform over a strip of 16.
#include <algorithm>

#include "f8_common.h"

namespace moe {

// Strips: a workgroup of four waves takes 16 weight rows (gate/up: 16 of
// each matrix) against up to 16 RB rows of one group, each wave every
// fourth block of K, operands straight from memory to registers (each
// weight code is used by one wave only); the four partial sums meet in LDS.
template <int MODE, int RB>
__global__ __launch_bounds__(256) void f8_strip_kernel(F8Args a) {
  constexpr int WF = MODE == 1 ? 2 : 1;
  __shared__ float part[3][WF][RB][256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, kq = (lane >> 4) * 32;
  const int K = a.K, N = a.N;
  const int nkb = (K + 127) / 128, nnb = (N + 127) / 128;
  const int strips = (N + 15) / 16;
  const int64_t groups = MODE == 0 ? (a.M + 16 * RB - 1) / (16 * RB) : a.meta[a.meta_index];
  const int64_t items = groups * strips;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t gi = it / strips;
    const int n0 = (int)(it - gi * strips) * 16;
    int64_t row0;
    int rows, e = 0;
    if (MODE == 0) {
      row0 = gi * 16 * RB;
      rows = (int)min((int64_t)(16 * RB), a.M - row0);
    } else {
      e = a.list[4 * gi];
      rows = a.list[4 * gi + 2];
      row0 = a.list[4 * gi + 3];
    }
    // past the last weight row or group row: the last one again, not stored
    const int n = min(n0 + lr, N - 1);
    const uint8_t* w[WF];
    const float* ws[WF];
#pragma unroll
    for (int f = 0; f < WF; ++f) {
      w[f] = (f ? a.B1 : a.B0) + ((size_t)e * N + n) * K;
      ws[f] = (f ? a.B1s : a.B0s) + ((size_t)e * nnb + (n0 >> 7)) * nkb;
    }
    const uint8_t* x[RB];
    const float* xs[RB];
#pragma unroll
    for (int t = 0; t < RB; ++t) {
      int64_t r = row0 + min(16 * t + lr, rows - 1);
      if (MODE == 1) r = a.pair_token[r];
      x[t] = a.A + (size_t)r * K;
      xs[t] = a.As + (size_t)r * nkb;
    }
    floatx4 acc[WF][RB];
#pragma unroll
    for (int f = 0; f < WF; ++f)
#pragma unroll
      for (int t = 0; t < RB; ++t) acc[f][t] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int kb = wave; kb < nkb; kb += 4) {
      const int k = kb * 128 + kq;
      v8i32 wv[WF], xv[RB];
#pragma unroll
      for (int f = 0; f < WF; ++f) wv[f] = load_codes(w[f], k, K);
#pragma unroll
      for (int t = 0; t < RB; ++t) xv[t] = load_codes(x[t], k, K);
      Codes wc[WF];
#pragma unroll
      for (int f = 0; f < WF; ++f) wc[f] = widen(wv[f]);
#pragma unroll
      for (int t = 0; t < RB; ++t) {
        const float sx = xs[t][kb];
        const Codes xc = widen(xv[t]);
#pragma unroll
        for (int f = 0; f < WF; ++f) {
          const floatx4 p = block_product(wc[f], xc);
          const float sc = sx * ws[f][kb];
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[f][t][q] = fmaf(p[q], sc, acc[f][t][q]);
        }
      }
    }
    if (wave) {
#pragma unroll
      for (int f = 0; f < WF; ++f)
#pragma unroll
        for (int t = 0; t < RB; ++t)
          *reinterpret_cast<floatx4*>(&part[wave - 1][f][t][lane * 4]) = acc[f][t];
    }
    __syncthreads();
    if (!wave) {
#pragma unroll
      for (int t = 0; t < RB; ++t) {
#pragma unroll
        for (int f = 0; f < WF; ++f)
#pragma unroll
          for (int s = 0; s < 3; ++s)
            acc[f][t] += *reinterpret_cast<floatx4*>(&part[s][f][t][lane * 4]);
        const int r = 16 * t + lr;
        if (r >= rows) continue;
        const int nc = n0 + (lane >> 4) * 4;
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v[q] = MODE == 1 ? swiglu(acc[0][t][q], acc[WF - 1][t][q], a.clamp) : acc[0][t][q];
        const size_t at = (size_t)(row0 + r) * N + nc;
        if (MODE != 0 || (N & 3) == 0) {
          if (nc < N) store_out4(a.out, MODE == 1 ? MOE_F32 : a.odt, at, v);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (nc + q < N) store_out1(a.out, a.odt, at + q, v[q]);
        }
      }
    }
    __syncthreads();
  }
}

hipError_t launch_f8_strip(const F8Args& a, int rb, int ncu, hipStream_t s) {
  const int64_t groups = a.mode == 0 ? (a.M + 16 * rb - 1) / (16 * rb) : a.max_groups;
  const int64_t items = groups * ((a.N + 15) / 16);
  if (items == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>(items, (int64_t)ncu * 16)), block(256);
  if (rb == 1) {
    if (a.mode == 0) hipLaunchKernelGGL((f8_strip_kernel<0, 1>), grid, block, 0, s, a);
    else if (a.mode == 1) hipLaunchKernelGGL((f8_strip_kernel<1, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((f8_strip_kernel<2, 1>), grid, block, 0, s, a);
  } else {
    if (a.mode == 0) hipLaunchKernelGGL((f8_strip_kernel<0, 4>), grid, block, 0, s, a);
    else if (a.mode == 1) hipLaunchKernelGGL((f8_strip_kernel<1, 4>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((f8_strip_kernel<2, 4>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
