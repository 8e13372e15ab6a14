// Device helpers of the row-wise kernels (quantisers and norms): eight
// consecutive values of a tensor whose type is known at run time, block
// scales of the 8-bit format, sums over the threads of a row.
#pragma once

#include "device_common.h"
#include "f8_internal.h"

namespace moe {

// A launch holds fewer than 2^32 threads along x: more than 2^20 workgroups
// go into rows of that many, and a kernel asks for its number here (those
// past the last return).
inline dim3 wide_grid(int64_t n) {
  const unsigned x = (unsigned)(n < (1 << 20) ? n : 1 << 20);
  return dim3(x, (unsigned)((n + x - 1) / x));
}
__device__ __forceinline__ uint32_t wide_block() { return blockIdx.y * gridDim.x + blockIdx.x; }

// 8 values as loaded: f32 fills both words, 16-bit types the first. The type
// is uniform over a launch, so the branches are scalar.
struct Raw8 { uint4 a, b; };

__device__ __forceinline__ Raw8 load_raw8(const void* base, int dt, size_t idx) {
  Raw8 r;
  if (dt == MOE_F32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + idx);
    r.a = p[0];
    r.b = p[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + idx);
    r.b = uint4{0u, 0u, 0u, 0u};
  }
  return r;
}

__device__ __forceinline__ void raw8_to_f32(const Raw8& r, int dt, float (&v)[8]) {
  if (dt == MOE_F32) {
    v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
    v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
    v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
    v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
  } else if (dt == MOE_BF16) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const half8 h = __builtin_bit_cast(half8, r.a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  }
}

// one rounding (to nearest, ties to even) of each f32 value to the type
__device__ __forceinline__ void store8(void* base, int dt, size_t idx, const float (&v)[8]) {
  if (dt == MOE_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + idx);
    p[0] = float4{v[0], v[1], v[2], v[3]};
    p[1] = float4{v[4], v[5], v[6], v[7]};
  } else if (dt == MOE_BF16) {
    bf16x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
    *reinterpret_cast<bf16x8*>(static_cast<uint16_t*>(base) + idx) = o;
  } else {
    half8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (_Float16)v[i];
    *reinterpret_cast<half8*>(static_cast<uint16_t*>(base) + idx) = o;
  }
}

// ---- 8-bit blocks -----------------------------------------------------------
//
// A block of values with largest magnitude m has a = max(m, 2^-100), scale
// s = a / 448 and codes q = e4m3(v * (448 / a)); 448 is the format's largest
// value, so |v * (448 / a)| rounds to at most 448 and never overflows. Both
// quotients are correctly rounded f32 divisions and the product is one f32
// rounding: 16-bit values often fall halfway between two codes, so a
// quotient off by one unit would give other codes. Magnitudes are compared
// as integers, which orders a NaN above infinity: a block holding either
// gets a scale of infinity or NaN and dequantises to NaN.
constexpr float kF8Max = 448.f;
constexpr float kF8Tiny = 0x1p-100f;

__device__ __forceinline__ uint32_t mag_bits(float v) {
  return __float_as_uint(v) & 0x7FFFFFFFu;
}

__device__ __forceinline__ uint32_t mag_max8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag_bits(v[i]));
  return m;
}

struct F8Scale { float s, inv; };
__device__ __forceinline__ F8Scale f8_scale(uint32_t mag) {
  float a = __uint_as_float(mag);
  a = a < kF8Tiny ? kF8Tiny : a;
  return {a / kF8Max, kF8Max / a};
}

// 8 codes of v * inv, lowest byte first
__device__ __forceinline__ uint2 f8_pack8(const float (&v)[8], float inv) {
  uint32_t o[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w, true);
    o[h] = (uint32_t)w;
  }
  return uint2{o[0], o[1]};
}

// Lane exchanges within a row of 16 lanes by DPP (a few cycles; a shuffle
// goes through the LDS): neighbours, pairs, mirrored halves, mirrored row.
// After the four every lane holds the row's result.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// the largest magnitude over 16 neighbouring lanes (16 x 8 values: a block)
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = max(m, dpp<kDppXor1>(m));
  m = max(m, dpp<kDppXor2>(m));
  m = max(m, dpp<kDppHalfMirror>(m));
  return max(m, dpp<kDppMirror>(m));
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<kDppXor1>(v);
  v = dpp_add<kDppXor2>(v);
  v = dpp_add<kDppHalfMirror>(v);
  v = dpp_add<kDppMirror>(v);
  auto row = [&](int r) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16 * r));
  };
  return (row(0) + row(1)) + (row(2) + row(3));
}

// Sums of N values over the TPR threads of a row, the same bits in every
// thread. sh: the row group's own N * TPR / 64 floats, used once between
// barriers (the caller alternates between two). Every thread of the
// workgroup takes part.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* sh) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = (threadIdx.x % TPR) >> 6, lane = threadIdx.x & 63;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) sh[i * W + wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += sh[i * W + w];
      v[i] = s;
    }
  }
}

}  // namespace moe
