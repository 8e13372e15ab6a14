// Products on 8-bit blocks on gfx950: e4m3 rows with a scale per row and
// 128 values times e4m3 weights with a scale per 128 x 128 block.
//
//   out[row, n] = sum_b As[row, b] Bs[n / 128, b] (sum_{k in b} A[row, k] B[n, k])
//
// The codes become f16 on the way to the matrix units, exactly (e4m3 has
// fewer exponent and fraction bits), and four v_mfma 16x16x32 sum a block of
// 128 in f32. (The 8-bit matrix instructions align the products they add to
// the largest and drop what lies 2^-14 below it: with a zero elsewhere,
// 256 * 256 + 2 * 2 sums to 65536. The 16-bit ones keep f32's 24 bits.) The
// block's sum is scaled and added to the f32 accumulator, one fma a value.
// The weights are the matrix instruction's first operand and the rows its
// second, so a lane holds four neighbouring outputs of one row and the row's
// scale, and the weights' scale is uniform over a strip of 16.
#include <algorithm>

#include "device_common.h"

namespace moe {

typedef int v8i32 __attribute__((ext_vector_type(8)));

// 8 codes (two words) as f16
__device__ __forceinline__ half8 codes_f16(int lo, int hi) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
  const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
  const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
  const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
  return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A lane's 32 codes of a block as the four steps' operands. A step takes 8
// codes of each of the four lane groups; both operands take the same ones,
// so the order of K within a block does not matter.
struct Codes { half8 h[4]; };
__device__ __forceinline__ Codes widen(const v8i32& v) {
  Codes c;
#pragma unroll
  for (int s = 0; s < 4; ++s) c.h[s] = codes_f16(v[2 * s], v[2 * s + 1]);
  return c;
}

__device__ __forceinline__ floatx4 block_product(const Codes& a, const Codes& b) {
  floatx4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; ++s) p = mfma16(a.h[s], b.h[s], p);
  return p;
}

// 32 codes of a row from k: two 16-byte pieces, zeros past the row's end (a
// row ends on a piece, K being a multiple of 16).
__device__ __forceinline__ v8i32 load_codes(const uint8_t* row, int k, int K) {
  uint4 lo = {0u, 0u, 0u, 0u}, hi = lo;
  if (k < K) lo = ldg16(row + k);
  if (k + 16 < K) hi = ldg16(row + k + 16);
  return v8i32{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

__device__ __forceinline__ void store_out4(void* out, int dt, size_t at, const float (&v)[4]) {
  if (dt == MOE_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = float4{v[0], v[1], v[2], v[3]};
  } else if (dt == MOE_BF16) {
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<b4*>(static_cast<__bf16*>(out) + at) =
        b4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
  } else {
    typedef _Float16 h4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<h4*>(static_cast<_Float16*>(out) + at) =
        h4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
  }
}

__device__ __forceinline__ void store_out1(void* out, int dt, size_t at, float v) {
  if (dt == MOE_F32) static_cast<float*>(out)[at] = v;
  else if (dt == MOE_BF16) static_cast<__bf16*>(out)[at] = (__bf16)v;
  else static_cast<_Float16*>(out)[at] = (_Float16)v;
}

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
