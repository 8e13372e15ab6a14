// Products of up to 16 rows of x with a stream of weight rows, on the 16-bit
// matrix instructions: fragments of x held in registers, blocks of 128 values
// of 16 weight rows as loaded, 4-bit codes widened exactly.
//
// One matrix instruction takes 16 rows of x (its A operand; lane l: row l & 15,
// values 8 (l >> 4) .. + 7 of the step's 32) and 16 weight rows (B operand, lane
// l: row l & 15, the same values) and adds into D, whose element i of lane l is
// row 4 (l >> 4) + i of A against row l & 15 of B. Token t sits in A's row
// 4 (t & 3) + (t >> 2): tokens 4 i .. 4 i + 3 are then element i of the four lane
// groups, and up to 4 NI tokens use the first NI elements only.
//
// 4-bit codes are not rounded to 16-bit weights: a code is ORed below a constant
// exponent (f16 64 + c, bf16 128 + c for c = 0..15, exact), one instruction sums
// one step of 32 values, a group or half of one, and that sum is scaled in f32.
// The constant's share, off * sum of the step's x, is the instruction's starting
// accumulator: -off * sum x, made once per fragment of x by an instruction
// against a constant B. Seven integer operations a word of eight codes (three
// shifts, four three-input logic operations), a lane exchange a word and NI fma a
// step; widening to fp16 weights takes 16 and more.
#pragma once

#include "device_common.h"

namespace moe {

// The 16-bit types: widening of codes, vectors, the lanes' constants.
template <class S> struct R16;
template <> struct R16<_Float16> {
  using V = half8;
  static constexpr float kOff = 64.f;               // 0x5400: units of 2^-4, codes from bit 4
  static constexpr uint32_t kBase = 0x54005400u, kMask = 0x00F000F0u;
  static constexpr int kFlip = 7;                   // the codes' top bit
  // word -> the nibbles (i, i + 4) at the mask's place
  template <int I> static __device__ __forceinline__ uint32_t place(uint32_t w) {
    return I == 0 ? w << 4 : w >> (4 * I - 4);
  }
};
template <> struct R16<__bf16> {
  using V = bf16x8;
  static constexpr float kOff = 128.f;              // 0x4300: units of 1
  static constexpr uint32_t kBase = 0x43004300u, kMask = 0x000F000Fu;
  static constexpr int kFlip = 3;
  template <int I> static __device__ __forceinline__ uint32_t place(uint32_t w) {
    return w >> (4 * I);
  }
};

// What a signed code's widened value exceeds it by (its nibble is flipped to
// code + 8), and an unsigned one's.
template <class S, int FMT> constexpr float kQ4Off = R16<S>::kOff + (FMT == 0 ? 8.f : 0.f);

// Eight codes of a word as off + code, in the order 0 4 1 5 2 6 3 7.
template <class S, int FMT>
__device__ __forceinline__ typename R16<S>::V q4_widen(uint32_t w) {
  using R = R16<S>;
  constexpr uint32_t c = R::kBase | (FMT == 0 ? 0x00010001u << R::kFlip : 0u);
  // (w & mask) ^ c
  uint4 o;
  o.x = __builtin_amdgcn_bitop3_b32(R::template place<0>(w), R::kMask, c, 0x6A);
  o.y = __builtin_amdgcn_bitop3_b32(R::template place<1>(w), R::kMask, c, 0x6A);
  o.z = __builtin_amdgcn_bitop3_b32(R::template place<2>(w), R::kMask, c, 0x6A);
  o.w = __builtin_amdgcn_bitop3_b32(R::template place<3>(w), R::kMask, c, 0x6A);
  return __builtin_bit_cast(typename R::V, o);
}

// Eight values of x in the codes' order.
__device__ __forceinline__ uint4 q4_order(uint4 v) {
  uint4 o;
  o.x = __builtin_amdgcn_perm(v.z, v.x, 0x05040100u);   // 0 4
  o.y = __builtin_amdgcn_perm(v.z, v.x, 0x07060302u);   // 1 5
  o.z = __builtin_amdgcn_perm(v.w, v.y, 0x05040100u);   // 2 6
  o.w = __builtin_amdgcn_perm(v.w, v.y, 0x07060302u);   // 3 7
  return o;
}

// Word j of lane group g to word g of lane group j (groups of 16 lanes).
__device__ __forceinline__ uint4 lane_group_transpose(uint4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return uint4{c[0], c[1], d[0], d[1]};
}

// A block of 128 values of 16 rows, as loaded. FMT -1: 16-bit weights.
template <int FMT> struct WBlock {
  uint4 q;
  uint32_t p[FMT == 1 ? 4 : 2];
};
template <> struct WBlock<-1> { uint4 q[4]; };

// A lane's weight row: its first byte and its parameters' first byte.
struct WRow { const char* q; const char* p; };

// Row n of a [rows, K] matrix of format FMT.
template <int FMT>
__device__ __forceinline__ WRow weight_row(const void* data, const void* params, size_t n, int K) {
  if constexpr (FMT < 0) return {(const char*)data + n * (size_t)K * 2, nullptr};
  else return {(const char*)data + n * (size_t)(K / 2),
               (const char*)params + n * (size_t)(K / Q4F<FMT>::kGroup) * Q4F<FMT>::kPB};
}

// Block kb (values 128 kb ..) of the lane's row. Lane group g loads bytes 16 g
// of each 64. RAGGED: K is no multiple of 128, and pieces of 32 values behind
// the row's last (pieces = K / 32) are read from the last with parameters of
// zero (x's fragments are zero there).
template <int FMT, bool RAGGED>
__device__ __forceinline__ WBlock<FMT> load_wblock(const WRow& r, int kb, int pieces) {
  const int g = (threadIdx.x >> 4) & 3;
  WBlock<FMT> b;
  if constexpr (FMT < 0) {
    static_assert(!RAGGED, "16-bit weights come in whole blocks");
#pragma unroll
    for (int i = 0; i < 4; ++i) b.q[i] = ldg16(r.q + (size_t)kb * 256 + 64 * i + 16 * g);
  } else {
    using Q = Q4F<FMT>;
    constexpr int kP = FMT == 1 ? 4 : 2;
    const int piece = 4 * kb + g;
    b.q = ldg16(r.q + (size_t)(RAGGED ? min(piece, pieces - 1) : piece) * 16);
    const char* p = r.p + (size_t)kb * (128 / Q::kGroup) * Q::kPB;
    if (!RAGGED || 4 * kb + 4 <= pieces) {
      // rows of an odd number of parameters start on two or four bytes
      if constexpr (RAGGED) __builtin_memcpy(b.p, p, 4 * kP);
      else __builtin_memcpy(b.p, __builtin_assume_aligned(p, 4), 4 * kP);
    } else {
      const int left = pieces - 4 * kb;   // 1 .. 3 pieces
#pragma unroll
      for (int i = 0; i < kP; ++i) b.p[i] = 0u;
      if constexpr (FMT == 0) {
        for (int i = 0; i < left; ++i) {
          const uint32_t s = *reinterpret_cast<const uint16_t*>(p + 2 * i);
          if (i < 2) b.p[0] |= s << (16 * i);
          else b.p[1] = s;
        }
      } else {
        // a64 rows are whole pairs of pieces
        const int n = FMT == 1 ? left : left / 2;
#pragma unroll
        for (int i = 0; i < kP; ++i)
          if (i < n) b.p[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
      }
    }
  }
  return b;
}

// Fragments of x over a block of 128 values (4 steps), and for 4-bit weights
// -off * (sum of each step's x) of the lane's tokens.
template <class S, int FMT> struct XBlock {
  typename R16<S>::V v[4];
  floatx4 c[FMT < 0 ? 1 : 4];
};

// x16(step): the lane's eight values of a step (zero past K), in order.
template <class S, int FMT, class F>
__device__ __forceinline__ XBlock<S, FMT> make_xblock(F&& x16) {
  using V = typename R16<S>::V;
  XBlock<S, FMT> b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = x16(i);
    if constexpr (FMT < 0) {
      b.v[i] = as_v8<V>(v);
    } else {
      b.v[i] = as_v8<V>(q4_order(v));
      V k;
#pragma unroll
      for (int j = 0; j < 8; ++j) k[j] = (S)(-kQ4Off<S, FMT>);
      b.c[i] = mfma16(b.v[i], k, floatx4{0.f, 0.f, 0.f, 0.f});
    }
  }
  return b;
}

__device__ __forceinline__ float half_lo(uint32_t w) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)w);
}
__device__ __forceinline__ float half_hi(uint32_t w) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
}

// acc[i] += the block's products of the lane's tokens 4 i + (lane >> 4) with
// its weight row.
template <class S, int FMT, int NI>
__device__ __forceinline__ void block_product(const XBlock<S, FMT>& x, const WBlock<FMT>& w,
                                              floatx4& acc) {
  using V = typename R16<S>::V;
  if constexpr (FMT < 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = mfma16(x.v[i], as_v8<V>(w.q[i]), acc);
  } else {
    const uint4 t = lane_group_transpose(w.q);
    const uint32_t words[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const floatx4 m = mfma16(x.v[i], q4_widen<S, FMT>(words[i]), x.c[i]);
      float s, b = 0.f;
      if constexpr (FMT == 0) {
        s = i & 1 ? half_hi(w.p[i / 2]) : half_lo(w.p[i / 2]);
      } else {
        const uint32_t sb = w.p[FMT == 1 ? i : i / 2];
        s = half_lo(sb);
        b = half_hi(sb) * (-1.f / kQ4Off<S, FMT>);   // c holds -off sum x; exact
      }
#pragma unroll
      for (int e = 0; e < NI; ++e) {
        acc[e] = fmaf(s, m[e], acc[e]);
        if constexpr (FMT != 0) acc[e] = fmaf(b, x.c[i][e], acc[e]);
      }
    }
  }
}

}  // namespace moe
