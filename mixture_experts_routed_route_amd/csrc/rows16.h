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
// exponent (16 + c for c = 0..15, exact), one instruction sums one step of 32
// values, a group or half of one, and that sum is scaled in f32. The constant's
// share, off * sum of the step's x, is the instruction's starting accumulator:
// -off * sum x, made once per fragment of x by an instruction against a constant
// B. 16 is the least power of two whose significand holds a code: what it adds to
// a sum's rounding grows with it (rows of one sign, K 4096: 4e-7 to 1.6e-6 with 64 +
// c and 128 + c, which need a shift less, 6e-8 to 3e-7 so). Eight
// integer operations a word of eight codes (four shifts, four three-input logic
// operations), a lane exchange a word and NI fma a step; widening to fp16 weights
// takes 16 and more.
#pragma once

#include "device_common.h"
#include "q4_addr.h"

namespace moe {

// The 16-bit types: widening of codes, vectors, the lanes' constants.
template <class S> struct R16;
template <> struct R16<_Float16> {
  using V = half8;
  static constexpr uint32_t kBase = 0x4C004C00u, kMask = 0x03C003C0u;   // codes from bit 6
  static constexpr int kFlip = 9;                                       // their top bit
  // word -> the nibbles (i, i + 4) at the mask's place
  template <int I> static __device__ __forceinline__ uint32_t place(uint32_t w) {
    return I < 2 ? w << (6 - 4 * I) : w >> (4 * I - 6);
  }
};
template <> struct R16<__bf16> {
  using V = bf16x8;
  static constexpr uint32_t kBase = 0x41804180u, kMask = 0x00780078u;   // codes from bit 3
  static constexpr int kFlip = 6;
  template <int I> static __device__ __forceinline__ uint32_t place(uint32_t w) {
    return I < 1 ? w << 3 : w >> (4 * I - 3);
  }
};

// What a signed code's widened value exceeds it by (its nibble is flipped to
// code + 8), and an unsigned one's.
template <class S, int FMT> constexpr float kQ4Off = FMT == 0 ? 24.f : 16.f;

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

// A block of 128 values of 16 rows, as loaded. FMT -1: 16-bit weights, lane l of
// load i the values 32 i + 8 (l >> 4) .. of row l & 15, as the matrix instruction
// takes them. 4-bit: lane l the 32 codes ("piece") l & 3 of row l >> 2, so that
// neighbouring lanes read neighbouring bytes (the cache takes one access for 64
// such bytes, not four; with a row a lane its accesses bound the stream at 3.5
// TB/s), and in lanes 0 .. 15 the parameters of row l.
template <int FMT> struct WBlock {
  uint4 q;
  uint32_t p[FMT == 1 ? 4 : 2];
};
template <> struct WBlock<-1> { uint4 q[4]; };

// Where a row's length leaves the last block short: not at all (K a multiple of
// 128); rows of whole 4-byte words of parameters; rows of an odd number of 2-byte
// scales.
enum Ragged : int { kWhole = 0, kWords = 1, kOdd = 2 };

// 16 weight rows: descriptors of their bytes and parameters (scalar) and the
// lane's place in them. Rows past the matrix's last (and blocks past the end, see
// load_wblock) read as zeros, without a memory access.
template <int FMT> struct WStrip {
  __amdgpu_buffer_rsrc_t q, p;
  const char* prow;          // kOdd: the lane's row of parameters
  uint32_t vq, vp, vr;       // vp: parameters a block, vr: a run (load_params)
};

__device__ __forceinline__ uint4 buffer16(__amdgpu_buffer_rsrc_t r, uint32_t v, uint32_t s) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, v, s, 0));
}
__device__ __forceinline__ uint2 buffer8(__amdgpu_buffer_rsrc_t r, uint32_t v, uint32_t s) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, v, s, 0));
}

__device__ __forceinline__ uint4 buffer16(__amdgpu_buffer_rsrc_t r, LoadAt at) { return buffer16(r, at.v, at.s); }
__device__ __forceinline__ uint2 buffer8(__amdgpu_buffer_rsrc_t r, LoadAt at) { return buffer8(r, at.v, at.s); }
constexpr LoadAt kNoLoad = {kPastEnd, 0u};

// Rows n0 .. of the matrix [N, K] at data / params.
template <int FMT, int RAGGED>
__device__ __forceinline__ WStrip<FMT> weight_strip(const void* data, const void* params, int64_t N,
                                                    int64_t n0, int K) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t rows = n0 >= N ? 0u : (uint32_t)(N - n0 < 16 ? N - n0 : 16);
  WStrip<FMT> r;
  const uint32_t rb = FMT < 0 ? (uint32_t)K * 2 : (uint32_t)K / 2;
  r.q = make_rsrc((const char*)data + n0 * (int64_t)rb, rows * rb);
  r.prow = nullptr;
  if constexpr (FMT < 0) {
    r.vq = (lane & 15) * rb + (lane >> 4) * 16u;
    r.vp = r.vr = 0;
    r.p = r.q;
  } else {
    using Q = Q4F<FMT>;
    const uint32_t pb = (uint32_t)(K / Q::kGroup) * Q::kPB;
    const char* p = (const char*)params + n0 * (int64_t)pb;
    r.vq = codes_start(lane, rb);
    r.p = make_rsrc(p, rows * pb);
    r.vp = params_start(lane, pb);
    r.vr = run_start(lane, pb);
    if constexpr (RAGGED == kOdd)   // rows past the last read the matrix's first
      r.prow = (lane & 15) < rows ? p + (size_t)(lane & 15) * pb : (const char*)params;
  }
  return r;
}

// Block kb (values 128 kb ..) of the strip; kb >= end gives zeros. In a short last
// block the pieces behind the row's end have parameters of zero (their codes are the
// next row's, or zeros behind the last row; x's fragments are zero there).
template <int FMT, int RAGGED, bool PARAMS = true>
__device__ __forceinline__ WBlock<FMT> load_wblock(const WStrip<FMT>& r, int kb, int end, int K) {
  WBlock<FMT> b;
  if constexpr (FMT < 0) {
    static_assert(RAGGED == kWhole, "16-bit weights come in whole blocks");
    const uint32_t at = (uint32_t)(kb < end ? kb : 0);
    const uint32_t v = kb < end ? r.vq : kPastEnd;
#pragma unroll
    for (int i = 0; i < 4; ++i) b.q[i] = buffer16(r.q, v + 64u * i, at * 256u);
  } else {
    using Q = Q4F<FMT>;
    constexpr uint32_t kPer = 128 / Q::kGroup * Q::kPB;
    b.q = buffer16(r.q, kb < end ? codes_at(r.vq, kb, RAGGED == kWhole) : kNoLoad);
    if constexpr (!PARAMS) {
    } else if constexpr (RAGGED != kOdd) {
      const LoadAt at = kb < end ? params_at(r.vp, kb, kPer, RAGGED == kWhole) : kNoLoad;
      if constexpr (FMT == 1) {
        const uint4 w = buffer16(r.p, at);
        b.p[0] = w.x; b.p[1] = w.y; b.p[2] = w.z; b.p[3] = w.w;
      } else {
        const uint2 w = buffer8(r.p, at);
        b.p[0] = w.x; b.p[1] = w.y;
      }
    } else {
      static_assert(RAGGED != kOdd || FMT == 0, "only scales alone have two bytes");
      const int left = kb < end ? K / 32 - 4 * kb : 0;   // pieces
      const char* p = r.prow + (size_t)(kb < end ? kb : 0) * kPer;
      b.p[0] = b.p[1] = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left)
          b.p[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + 2 * i) << (16 * (i & 1));
    }
  }
  return b;
}

// Parameters of kRun blocks from block kb on, as loaded: lane 4 r + q has 16 bytes of
// row r. A run's bytes are asked for at once: 8 bytes a row and block would be a
// request each. What lies behind the row (its next row, or zeros behind the strip's
// last) is not used.
template <int FMT> constexpr int kRun = FMT == 1 ? 4 : 8;

template <int FMT>
__device__ __forceinline__ uint4 load_params(const WStrip<FMT>& r, int kb, int end) {
  using Q = Q4F<FMT>;
  return buffer16(r.p, kb < end ? run_at(r.vr, kb, 128 / Q::kGroup * Q::kPB) : kNoLoad);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Block i of the run (a constant) for the lane's row (lane & 15).
template <int FMT>
__device__ __forceinline__ void run_params(const uint4& p, int i, uint32_t* out) {
  const int row = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int k = 0; k < (FMT == 1 ? 4 : 2); ++k)
    out[k] = (uint32_t)__builtin_amdgcn_ds_bpermute(
        (row + (FMT == 1 ? i : i >> 1)) * 4, (int)word_of(p, FMT == 1 ? k : (i & 1) * 2 + k));
}

// Fragments of x over a block of 128 values (4 steps), and for 4-bit weights
// -off * (sum of each step's x) of the lane's tokens.
template <class S, int FMT> struct XBlock {
  typename R16<S>::V v[4];
  floatx4 c[FMT < 0 ? 1 : 4];
};

// -off * the sum over a step's values, of every token
template <class S, int FMT>
__device__ __forceinline__ floatx4 x_constant(typename R16<S>::V v, floatx4 c) {
  typename R16<S>::V k;
#pragma unroll
  for (int j = 0; j < 8; ++j) k[j] = (S)(-kQ4Off<S, FMT>);
  return mfma16(v, k, c);
}

// The token in row lane & 15 of a fragment.
__device__ __forceinline__ int fragment_token() {
  return (threadIdx.x & 3) * 4 + ((threadIdx.x >> 2) & 3);
}

// x of up to 16 tokens over K values in LDS, for all waves of a workgroup: rows of
// K values and 16 bytes (so that 16 rows at one place lie in different banks),
// in the codes' order for 4-bit weights, then their constants, 16 floats a step.
template <int FMT>
constexpr size_t x_lds_bytes(int T, int K) {
  return (size_t)T * (K * 2 + 16) + (FMT < 0 ? 0 : (size_t)K / 32 * 64);
}

// Values k0 .. k0 + KL of rows of x (K values apart; zeros from K on), KL a
// multiple of 128. The caller waits at a barrier.
template <class S, int FMT>
__device__ __forceinline__ void stage_x(char* lds, const S* x, int T, int k0, int KL, int K) {
  using V = typename R16<S>::V;
  constexpr int kAhead = 4;   // loads in flight
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int tok = fragment_token(), steps = KL / 32, stride = KL * 2 + 16;
  const auto rsrc = make_rsrc(x, (uint32_t)T * (uint32_t)K * 2u);
  float* c = (float*)(lds + (size_t)T * stride);
  for (int f0 = wave; f0 < steps; f0 += waves * kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = k0 + 32 * (f0 + i * waves) + (lane >> 4) * 8;
      // lanes without a token, and values behind the row, read zeros
      v[i] = buffer16(rsrc, tok < T && k < K ? (uint32_t)(tok * K + k) * 2u : kPastEnd, 0);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int f = f0 + i * waves;
      if (f >= steps) break;
      if constexpr (FMT >= 0) {
        v[i] = q4_order(v[i]);
        const floatx4 s = x_constant<S, FMT>(as_v8<V>(v[i]), floatx4{0.f, 0.f, 0.f, 0.f});
        if ((lane & 15) == 0) *reinterpret_cast<floatx4*>(c + f * 16 + (lane >> 4) * 4) = s;
      }
      if (tok < T) *reinterpret_cast<uint4*>(lds + tok * stride + f * 64 + (lane >> 4) * 16) = v[i];
    }
  }
}

// Block kb of the staged x; lanes of rows past T read the first. NI as below.
template <class S, int FMT, int NI>
__device__ __forceinline__ XBlock<S, FMT> x_block(const char* lds, int T, int KL, int kb) {
  using V = typename R16<S>::V;
  const int lane = threadIdx.x & 63, tok = fragment_token(), stride = KL * 2 + 16;
  const char* p = lds + (tok < T ? tok : 0) * stride + kb * 256 + (lane >> 4) * 16;
  const char* c = lds + (size_t)T * stride + kb * 256 + (lane >> 4) * 16;
  XBlock<S, FMT> b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b.v[i] = as_v8<V>(*reinterpret_cast<const uint4*>(p + 64 * i));
    if constexpr (FMT >= 0) {
      // elements from NI on go nowhere: whatever their registers hold
      floatx4 h;
      if constexpr (NI == 4) h = *reinterpret_cast<const floatx4*>(c + 64 * i);
#pragma unroll
      for (int e = 0; e < NI && NI < 4; ++e) h[e] = reinterpret_cast<const float*>(c + 64 * i)[e];
      b.c[i] = h;
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

// Lane l of 0 .. 15's value in lanes l, 16 + l, 32 + l and 48 + l.
__device__ __forceinline__ uint32_t lane_group_bcast(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_ds_bpermute((threadIdx.x & 15) * 4, (int)v);
}

// Lane 4 r + p's word to lane r + 16 p.
__device__ __forceinline__ uint4 rows_to_columns(uint4 v) {
  const int lane = threadIdx.x & 63, from = ((lane & 15) * 4 + (lane >> 4)) * 4;
  return uint4{(uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.x),
               (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.y),
               (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.z),
               (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.w)};
}

// A block's four steps of 4-bit weights, ready for the matrix instruction: words of
// eight codes (row lane & 15), parameters of the lane's row.
template <int FMT> struct Q4Steps {
  uint32_t word[4];
  uint32_t p[FMT == 1 ? 4 : 2];
  __device__ __forceinline__ float scale(int i) const {
    if constexpr (FMT == 0) return i & 1 ? half_hi(p[i / 2]) : half_lo(p[i / 2]);
    else return half_lo(p[FMT == 1 ? i : i / 2]);
  }
  __device__ __forceinline__ float bias(int i) const {
    static_assert(FMT != 0, "a signed code has no bias");
    return half_hi(p[FMT == 1 ? i : i / 2]);
  }
};

// Codes as loaded, parameters of the lane's row; left: pieces from the block's first
// to the row's end.
template <int FMT, int RAGGED>
__device__ __forceinline__ Q4Steps<FMT> q4_steps(uint4 codes, const uint32_t* params, int left) {
  Q4Steps<FMT> s;
  const uint4 t = lane_group_transpose(rows_to_columns(codes));
  s.word[0] = t.x; s.word[1] = t.y; s.word[2] = t.z; s.word[3] = t.w;
#pragma unroll
  for (int i = 0; i < (FMT == 1 ? 4 : 2); ++i) {
    s.p[i] = params[i];
    if constexpr (RAGGED == kWords)
      if ((FMT == 1 ? i : 2 * i) >= left) s.p[i] = 0u;
  }
  return s;
}

// a block's parameters as load_wblock reads them, for the lane's row
template <int FMT, int RAGGED>
__device__ __forceinline__ void block_params(const WBlock<FMT>& w, uint32_t* out) {
#pragma unroll
  for (int i = 0; i < (FMT == 1 ? 4 : 2); ++i) out[i] = RAGGED == kOdd ? w.p[i] : lane_group_bcast(w.p[i]);
}

// acc[i] += the block's products of the lane's tokens 4 i + (lane >> 4), i < NI, with
// its weight row.
template <class S, int FMT, int NI>
__device__ __forceinline__ void block_product(const XBlock<S, FMT>& x, const Q4Steps<FMT>& q,
                                              floatx4& acc) {
  // two matrix instructions before the sums of the first are needed
#pragma unroll
  for (int h = 0; h < 4; h += 2) {
    floatx4 m[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i] = mfma16(x.v[h + i], q4_widen<S, FMT>(q.word[h + i]), x.c[h + i]);
#pragma unroll
    for (int i = h; i < h + 2; ++i)
#pragma unroll
      for (int e = 0; e < NI; ++e) {
        acc[e] = fmaf(q.scale(i), m[i - h][e], acc[e]);
        // c holds -off sum x; the quotient is exact
        if constexpr (FMT != 0) acc[e] = fmaf(q.bias(i) * (-1.f / kQ4Off<S, FMT>), x.c[i][e], acc[e]);
      }
  }
}

// A wave's stream: blocks first .. end - 1 of MATS strips against the staged x
// (whose block 0 is block k0b of the rows), kDepth blocks of each strip in flight.
// A block of 4-bit codes is half a cache line of each row: two are asked for back to
// back, or the line would be fetched twice.
template <class S, int FMT, int NI, int MATS, int RAGGED> struct Stream {
  static constexpr bool kRuns = FMT >= 0 && RAGGED != kOdd;   // parameters by runs
  static constexpr int kPair = FMT < 0 ? 1 : 2;
  // as many as 128 registers a wave hold; beside them the two strips of gate and up spill
  // 8 or 9 of 9 .. 16 tokens on 4-bit weights and 3 of 5 .. 8 (groups of 32 with biases), one strip 3 of rows
  // with an odd number of scales
  static constexpr int kDepth = FMT < 0 ? 4 / MATS : MATS == 1 ? 8 : 4;
  static constexpr int kTurn = !kRuns ? kDepth : FMT == 1 ? (kDepth > 4 ? kDepth : 4) : 8;
  using Codes = WBlock<FMT>;
  Codes buf[kDepth][MATS];
  static constexpr int kR = kRuns ? kRun<FMT> : 8;   // blocks a run
  uint4 run_next[MATS];

  __device__ __forceinline__ void fill(const WStrip<FMT> (&m)[MATS], int i, int kb, int end, int K) {
#pragma unroll
    for (int j = 0; j < MATS; ++j)
#pragma unroll
      for (int h = 0; h < kPair; ++h)
        buf[i + h][j] = load_wblock<FMT, RAGGED, !kRuns>(m[j], kb + h, end, K);
  }
  __device__ __forceinline__ void start(const WStrip<FMT> (&m)[MATS], int first, int end, int K) {
    if constexpr (kRuns)
#pragma unroll
      for (int j = 0; j < MATS; ++j) run_next[j] = load_params<FMT>(m[j], first, end);
#pragma unroll
    for (int i = 0; i < kDepth; i += kPair) fill(m, i, first + i, end, K);
  }
  __device__ __forceinline__ void run(const WStrip<FMT> (&m)[MATS], const char* lds, int T, int KL, int k0b,
                                      int first, int end, int K, floatx4 (&acc)[MATS]) {
    for (int kb = first; kb < end; kb += kTurn) {
      uint4 params[MATS];
#pragma unroll
      for (int i = 0; i < kTurn; i += kPair) {
        if constexpr (kRuns) {
          if (i % kR == 0) {
#pragma unroll
            for (int j = 0; j < MATS; ++j) {
              params[j] = run_next[j];
              run_next[j] = load_params<FMT>(m[j], kb + i + kR, end);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < kPair; ++h) {
          if (kb + i + h >= end) break;
          const XBlock<S, FMT> x = x_block<S, FMT, NI>(lds, T, KL, kb + i + h - k0b);
#pragma unroll
          for (int j = 0; j < MATS; ++j) {
            const Codes& w = buf[(i + h) % kDepth][j];
            if constexpr (FMT < 0) {
#pragma unroll
              for (int s = 0; s < 4; ++s)
                acc[j] = mfma16(x.v[s], as_v8<typename R16<S>::V>(w.q[s]), acc[j]);
            } else {
              uint32_t p[FMT == 1 ? 4 : 2];
              if constexpr (kRuns) run_params<FMT>(params[j], (i + h) % kR, p);
              else block_params<FMT, RAGGED>(w, p);
              block_product<S, FMT, NI>(
                  x, q4_steps<FMT, RAGGED>(w.q, p, K / 32 - 4 * (kb + i + h)), acc[j]);
            }
          }
        }
        if (kb + i >= end) break;
        fill(m, i % kDepth, kb + i + kDepth, end, K);
      }
    }
  }
};

// A workgroup has kRowWaves waves; 1 << split of them share a strip's blocks: the
// most that still give each strip its waves at once.
constexpr int kRowWaves = 16;
__device__ __forceinline__ int wave_split(int64_t strips, int blocks, int workgroups) {
  int s = 0;
  while (s < 4 && (strips << (s + 1)) <= (int64_t)workgroups * kRowWaves && (2 << s) <= blocks) ++s;
  return s;
}

// The sums of the waves that share a strip, in the first of them (wave a multiple
// of share): part [waves][NI][64] of all waves, between barriers.
template <int NI>
__device__ __forceinline__ void add_shared(const float* part, int wave, int share, floatx4& acc) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int e = 0; e < NI; ++e) {
    float v[kRowWaves];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w)
      v[w] = w < share ? part[((wave + w) * NI + e) * 64 + lane] : 0.f;
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) acc[e] += v[w];
  }
}

}  // namespace moe
