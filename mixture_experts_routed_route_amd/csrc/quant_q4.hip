// Quantiser of the 4-bit formats on gfx950: one pass over the values, a group's
// extremes by lane exchanges, codes and parameters as the products read them.
#include "rows_common.h"
#include "q4_internal.h"

namespace moe {

namespace {

__device__ __forceinline__ float dpp_f(float v, int which) {
  const uint32_t u = __float_as_uint(v);
  return __uint_as_float(which == 0 ? dpp<kDppXor1>(u) : which == 1 ? dpp<kDppXor2>(u)
                                                                     : dpp<kDppHalfMirror>(u));
}

// f32 to fp16, to nearest even, as bits
__device__ __forceinline__ uint32_t half_bits(float v) {
  return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// d / s rounded to f32, r = 1 / s rounded: a product and two of Markstein's corrections
// (IBM J. Res. Dev. 34, 1990). The first leaves less than a unit of the last place, the
// second the nearest value, as its remainder d - q s is exact: s has 11 bits and at least
// 2^-24; quotients so small that the remainder is not have the code 0 either way. Where
// infinities leave no remainder (inf - inf) the product is the answer: 0, inf or NaN.
// Fewer operations than a division's, all at the full rate: 65536 x 4096 fp16 values to
// scales alone 190 -> 166 us under the profiler (688 MB, 4.1 TB/s; 130 us at a copy's
// rate). Outside it a pass that decodes them too takes 269 us, less than the two kernels'
// traces (166 + 121).
__device__ __forceinline__ float quotient(float d, float s, float r) {
  const float q0 = d * r;
  const float q1 = __builtin_fmaf(__builtin_fmaf(-q0, s, d), r, q0);
  const float q2 = __builtin_fmaf(__builtin_fmaf(-q1, s, d), r, q1);
  return q2 == q2 ? q2 : q0;
}

// A thread owns 8 neighbouring values, a group is 4 (32 values) or 8 (64) lanes.
// The minimum and maximum keep a NaN, so that its group's scale is one. s = 0 (all
// values of a group equal, or too small for fp16) has codes of zero, and so has an
// infinite s (an infinity in the group, or values too far apart), whose values are NaN.
constexpr int kQ4Chunks = 4;   // loads in flight a thread
template <int FMT>
__global__ __launch_bounds__(256) void quant_q4_kernel(const void* __restrict__ w, int dt, int64_t n8,
                                                       uint32_t* __restrict__ data,
                                                       void* __restrict__ params) {
  constexpr int kLanes = Q4F<FMT>::kGroup / 8;
  const int64_t first = (int64_t)wide_block() * (256 * kQ4Chunks) + threadIdx.x;
  Raw8 raw[kQ4Chunks];
#pragma unroll
  for (int c = 0; c < kQ4Chunks; ++c) {
    const int64_t at = first + c * 256;
    if (at < n8) raw[c] = load_raw8(w, dt, (size_t)at * 8);
  }
#pragma unroll
  for (int c = 0; c < kQ4Chunks; ++c) {
    const int64_t at = first + c * 256;
    if (at >= n8) break;   // whole groups: n8 is a multiple of their lanes
    float v[8];
    raw8_to_f32(raw[c], dt, v);
    float hi, lo = 0.f;
    if constexpr (FMT == 0) {
      hi = __builtin_fabsf(v[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) hi = __builtin_elementwise_maximum(hi, __builtin_fabsf(v[i]));
    } else {
      hi = lo = v[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        hi = __builtin_elementwise_maximum(hi, v[i]);
        lo = __builtin_elementwise_minimum(lo, v[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < (kLanes == 8 ? 3 : 2); ++i) {
      hi = __builtin_elementwise_maximum(hi, dpp_f(hi, i));
      if constexpr (FMT != 0) lo = __builtin_elementwise_minimum(lo, dpp_f(lo, i));
    }
    const uint32_t sb = half_bits(FMT == 0 ? hi / 7.f : (hi - lo) / 15.f);
    const uint32_t bb = FMT == 0 ? 0u : half_bits(lo);
    const float s = (float)__builtin_bit_cast(_Float16, (uint16_t)sb);
    const float b = (float)__builtin_bit_cast(_Float16, (uint16_t)bb);
    constexpr float kMin = FMT == 0 ? -8.f : 0.f, kMax = FMT == 0 ? 7.f : 15.f;
    uint32_t word = 0u;
    const float r = 1.f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = FMT == 0 ? v[i] : v[i] - b;
      // fmin / fmax give the bound for a NaN: its group's scale is one, or infinite
      const float q = fminf(fmaxf(__builtin_rintf(quotient(d, s, r)), kMin), kMax);
      word |= ((uint32_t)(int)q & 15u) << (4 * i);
    }
    // zero times an infinite scale: a NaN, as any code times a NaN scale
    data[at] = s == 0.f || s == __builtin_inff() ? 0u : word;
    if (threadIdx.x % kLanes == 0) {
      const size_t g = (size_t)at / kLanes;
      if constexpr (FMT == 0) static_cast<uint16_t*>(params)[g] = (uint16_t)sb;
      else static_cast<uint32_t*>(params)[g] = sb | (bb << 16);
    }
  }
}

}  // namespace

hipError_t launch_quant_q4(const void* w, int dt, int fmt, int64_t rows, int64_t K, void* data,
                           void* params, hipStream_t s) {
  const int64_t n8 = rows * (K / 8);
  if (n8 == 0) return hipSuccess;
  const dim3 grid = wide_grid((n8 + 256 * kQ4Chunks - 1) / (256 * kQ4Chunks)), block(256);
  uint32_t* d = static_cast<uint32_t*>(data);
  if (fmt == 0) hipLaunchKernelGGL((quant_q4_kernel<0>), grid, block, 0, s, w, dt, n8, d, params);
  else if (fmt == 1) hipLaunchKernelGGL((quant_q4_kernel<1>), grid, block, 0, s, w, dt, n8, d, params);
  else hipLaunchKernelGGL((quant_q4_kernel<2>), grid, block, 0, s, w, dt, n8, d, params);
  return hipGetLastError();
}

}  // namespace moe
