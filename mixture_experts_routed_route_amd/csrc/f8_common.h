// Device helpers of the products on 8-bit blocks: operand fragments and
// output stores shared by the strip and the tile.
#pragma once

#include <type_traits>

#include "rows_common.h"

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

// A lane group's 32 codes of a block of a row: 16-byte pieces q and q + 4, so
// that the four groups read 64 neighbouring bytes at once. `row` points at
// piece q of the row's first block, k is the block's start; pieces past the
// row's end (a row ends on a piece, K being a multiple of 16) are zeros.
__device__ __forceinline__ v8i32 load_codes(const uint8_t* row, int q, int k, int K) {
  uint4 lo = {0u, 0u, 0u, 0u}, hi = lo;
  if (k + q * 16 < K) lo = ldg16(row + k);
  if (k + q * 16 + 64 < K) hi = ldg16(row + k + 64);
  return v8i32{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}
// the same within a whole block
__device__ __forceinline__ v8i32 load_codes(const uint8_t* at) {
  const uint4 lo = ldg16(at), hi = ldg16(at + 64);
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

// Both operands e4m3, without the hardware's block scales (zero operands
// select the instruction that has none). Its sum drops what lies 2^-13 below
// the largest of each eight products.
__device__ __forceinline__ floatx4 mfma_f8(v8i32 a, v8i32 b, floatx4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

}  // namespace moe
