// Products of more than 16 rows with 4-bit weights on gfx950: tiles of 16-row
// fragments of x against strips of 16 weight rows.
//
// As in rows16.h, a weight is never rounded: one matrix instruction a step of 32 values
// (two for groups of 64) on the codes, in bf16 as off + c from the accumulator -off *
// sum x, in fp16 as they are; its four sums a lane are scaled and added in f32. So an
// element costs one fma a group beside its multiplications, and a code's widening is
// shared by all rows of a tile: 128 rows a wave keep the vector units about as busy as
// the matrix units (a step of 128 x 64: 40 matrix instructions of 16 cycles in bf16, 32 in
// fp16 without biases, about 170 and 190 vector operations of 4).
// Weights rounded to 16 bits would cost neither the fma nor the constants, and an f32
// output its precision (2^-12 of fp16, 2^-9 of bf16 weights).
#include <type_traits>

#include "rows16.h"
#include "q4_internal.h"
#include "q4_tiles.h"

namespace moe {

namespace {

// Whether codes are widened without a constant: in fp16 a packed addition takes it away.
template <class S> constexpr bool kPlainCodes = std::is_same<S, _Float16>::value;

// Eight codes of a word in order (q4_widen's order would have x's values reordered in
// every fragment): bf16 off + code, ten operations, the code's bits below those of 16 in
// one byte; fp16 the code itself, thirteen, as 64 + c, whose code fills a byte's upper
// half, less 64.
template <class S, int FMT>
__device__ __forceinline__ typename R16<S>::V q4_widen_in_order(uint32_t w) {
  constexpr bool kHalf = kPlainCodes<S>;
  constexpr uint32_t mask = kHalf ? 0xF0F0F0F0u : 0x78787878u;
  constexpr uint32_t flip = (kHalf ? 0u : 0x80808080u) | (FMT != 0 ? 0u : kHalf ? 0x80808080u : 0x40404040u);
  const uint32_t lo = __builtin_amdgcn_bitop3_b32(w << (kHalf ? 4 : 3), mask, flip, 0x6A);      // 0 2 4 6
  const uint32_t hi = __builtin_amdgcn_bitop3_b32(kHalf ? w : w >> 1, mask, flip, 0x6A);        // 1 3 5 7
  const uint32_t p0 = __builtin_amdgcn_perm(hi, lo, 0x05010400u);   // 0 1 2 3
  const uint32_t p1 = __builtin_amdgcn_perm(hi, lo, 0x07030602u);   // 4 5 6 7
  constexpr uint32_t c = kHalf ? 0x54545454u : 0x41414141u;
  uint4 o;
  o.x = __builtin_amdgcn_perm(c, p0, 0x04010400u);
  o.y = __builtin_amdgcn_perm(c, p0, 0x04030402u);
  o.z = __builtin_amdgcn_perm(c, p1, 0x04010400u);
  o.w = __builtin_amdgcn_perm(c, p1, 0x04030402u);
  const auto v = __builtin_bit_cast(typename R16<S>::V, o);
  if constexpr (kHalf) return v - (_Float16)(FMT == 0 ? 72.f : 64.f);
  else return v;
}

// x staged as rows of 128 values, 16 pieces of 16 bytes; piece j of row r lies at place
// j ^ (r & 15), so that 16 neighbouring rows' pieces lie in different banks.
__device__ __forceinline__ int place(int row, int piece) { return row * 256 + ((piece ^ (row & 15)) * 16); }

// acc[m][s] += a block of MT x 16 rows of x (staged) against NS strips; left: pieces
// from the block's first to the row's end.
template <class S, int FMT, int RAGGED, int MT, int NS>
__device__ __forceinline__ void tile_block(const char* x, const WBlock<FMT> (&w)[NS], int left,
                                           floatx4 (&acc)[MT][NS]) {
  using V = typename R16<S>::V;
  constexpr int kG = FMT == 2 ? 2 : 1;   // steps a group
  const int lane = threadIdx.x & 63;
  Q4Steps<FMT> q[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    uint32_t p[FMT == 1 ? 4 : 2];
    block_params<FMT, RAGGED>(w[s], p);
    q[s] = q4_steps<FMT, kWhole>(w[s].q, p, 4);
  }
#pragma unroll
  for (int i = 0; i < 4; i += kG) {
    if (i >= left) break;
    V b[NS][kG];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int g = 0; g < kG; ++g) b[s][g] = q4_widen_in_order<S, FMT>(q[s].word[i + g]);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      V a[kG];
      floatx4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        a[g] = as_v8<V>(*reinterpret_cast<const uint4*>(
            x + place(m * 16 + (lane & 15), 4 * (i + g) + (lane >> 4))));
        if constexpr (FMT != 0 || !kPlainCodes<S>) c = x_constant<S, FMT>(a[g], c);
      }
      floatx4 d[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        d[s] = kPlainCodes<S> ? floatx4{0.f, 0.f, 0.f, 0.f} : c;
#pragma unroll
        for (int g = 0; g < kG; ++g) d[s] = mfma16(a[g], b[s][g], d[s]);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[m][s][e] = fmaf(q[s].scale(i), d[s][e], acc[m][s][e]);
          if constexpr (FMT != 0)
            acc[m][s][e] = fmaf(q[s].bias(i) * (-1.f / kQ4Off<S, FMT>), c[e], acc[m][s][e]);
        }
    }
  }
}

__device__ __forceinline__ void store_as(void* out, int odt, size_t at, float v) {
  if (odt == MOE_F32) static_cast<float*>(out)[at] = v;
  else if (odt == MOE_BF16) static_cast<__bf16*>(out)[at] = (__bf16)v;
  else static_cast<_Float16*>(out)[at] = (_Float16)v;
}

// ---- many rows ------------------------------------------------------------------
//
// 128 rows x 256 columns a workgroup of four waves side by side, two workgroups a
// compute unit; x by direct loads to LDS, a block of 128 values ahead, weights in
// registers a block ahead, one barrier a block.
constexpr int kStage = kTileM * 256;
static_assert(kTileM == 128 && kTileN == 4 * 64 && kTileThreads == 4 * 64, "four waves side by side");

// MT x 16 rows from m0 on
template <class S, int FMT, int RAGGED, int MT>
__device__ __forceinline__ void q4_tile(const RowsArgs& a, char* lds, int64_t m0, int64_t n0) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  n0 += wave * 64;
  const uint32_t rows = (uint32_t)(a.M - m0 < MT * 16 ? a.M - m0 : MT * 16), rb = (uint32_t)a.K * 2;
  // (its type by name: with auto the host pass drops the kernel without a word)
  const __amdgpu_buffer_rsrc_t rx = make_rsrc((const S*)a.x + m0 * a.K, rows * rb);
  const int blocks = (a.K + 127) / 128;
  WStrip<FMT> strip[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) strip[s] = weight_strip<FMT, RAGGED>(a.w, a.params, a.N, n0 + 16 * s, a.K);
  auto stage = [&](int kb, int buf) {
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int first = (wave * MT + j) * 4;   // the first of four rows
      const int row = first + (lane >> 4), piece = (lane & 15) ^ (row & 15);
      const uint32_t v = kb * 128 + piece * 8 < a.K ? (uint32_t)row * rb + piece * 16 : kPastEnd;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)(lds + buf * kStage + first * 256), 16, (int)v,
                                               kb * 256, 0, 0);
    }
  };
  floatx4 acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[m][s] = floatx4{0.f, 0.f, 0.f, 0.f};
  WBlock<FMT> next[4];
  stage(0, 0);
#pragma unroll
  for (int s = 0; s < 4; ++s) next[s] = load_wblock<FMT, RAGGED>(strip[s], 0, blocks, a.K);
  wait_vmcnt<0>();
  __syncthreads();
  for (int kb = 0; kb < blocks; ++kb) {
    WBlock<FMT> w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) w[s] = next[s];
    if (kb + 1 < blocks) {
      stage(kb + 1, (kb + 1) & 1);
#pragma unroll
      for (int s = 0; s < 4; ++s) next[s] = load_wblock<FMT, RAGGED>(strip[s], kb + 1, blocks, a.K);
    }
    tile_block<S, FMT, RAGGED, MT, 4>(lds + (kb & 1) * kStage, w, a.K / 32 - 4 * kb, acc);
    wait_vmcnt<0>();
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t row = m0 + m * 16 + (lane >> 4) * 4 + e;
      if (row < a.M) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int64_t n = n0 + s * 16 + (lane & 15);
          if (n < a.N) store_as(a.out, a.odt, (size_t)row * a.N + n, acc[m][s][e]);
        }
      }
    }
}

template <class S, int FMT, int RAGGED>
__global__ __launch_bounds__(kTileThreads, 2) void q4_tile_kernel(RowsArgs a, int tiles_n, int whole, int tiles) {
  extern __shared__ __attribute__((aligned(16))) char lds[];   // two blocks of x
  const TileAt t = tile_at((int)blockIdx.x, tiles_n, whole, tiles);
  if (t.rows == kTileM) q4_tile<S, FMT, RAGGED, 8>(a, lds, t.row, t.column);
  else if (t.rows) q4_tile<S, FMT, RAGGED, 4>(a, lds, t.row, t.column);
}

// ---- some rows --------------------------------------------------------------------
//
// MT x 16 rows x NS x 16 columns a workgroup, whose eight waves share K: each takes its
// own blocks of 128, with x's rows of the block in its own part of LDS (loaded a block
// ahead into registers), without a barrier until their sums meet.
constexpr int kSliceWaves = 8;

template <class S, int FMT, int RAGGED, int MT, int NS>
__global__ __launch_bounds__(64 * kSliceWaves) void q4_slice_kernel(RowsArgs a) {
  constexpr int kRows = MT * 16, kOut = MT * NS * 4;   // kOut: sums a lane
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char* mine = lds + wave * kRows * 256;
  const int64_t m0 = (int64_t)blockIdx.y * kRows, n0 = (int64_t)blockIdx.x * (NS * 16);
  const uint32_t rows = (uint32_t)(a.M - m0 < kRows ? a.M - m0 : kRows), rb = (uint32_t)a.K * 2;
  const auto rx = make_rsrc((const S*)a.x + m0 * a.K, rows * rb);
  const int blocks = (a.K + 127) / 128;
  const int first = blocks * wave / kSliceWaves, end = blocks * (wave + 1) / kSliceWaves;
  WStrip<FMT> strip[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) strip[s] = weight_strip<FMT, RAGGED>(a.w, a.params, a.N, n0 + 16 * s, a.K);
  floatx4 acc[MT][NS];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[m][s] = floatx4{0.f, 0.f, 0.f, 0.f};
  WBlock<FMT> next[NS];
  uint4 xn[MT * 4];
  auto load = [&](int kb) {
#pragma unroll
    for (int s = 0; s < NS; ++s) next[s] = load_wblock<FMT, RAGGED>(strip[s], kb, end, a.K);
    const int k = kb * 128 + (lane & 15) * 8;
#pragma unroll
    for (int j = 0; j < MT * 4; ++j)
      xn[j] = buffer16(rx, kb < end && k < a.K ? (uint32_t)(j * 4 + (lane >> 4)) * rb + (uint32_t)k * 2 : kPastEnd, 0);
  };
  load(first);
  for (int kb = first; kb < end; ++kb) {
    WBlock<FMT> w[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) w[s] = next[s];
#pragma unroll
    for (int j = 0; j < MT * 4; ++j)
      *reinterpret_cast<uint4*>(mine + place(j * 4 + (lane >> 4), lane & 15)) = xn[j];
    load(kb + 1);
    tile_block<S, FMT, RAGGED, MT, NS>(mine, w, a.K / 32 - 4 * kb, acc);
  }
  __syncthreads();   // x's part of LDS is free
  float* part = (float*)lds;   // [waves][kOut][64]
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[(wave * kOut + (m * NS + s) * 4 + e) * 64 + lane] = acc[m][s][e];
  __syncthreads();
  for (int o = wave; o < kOut; o += kSliceWaves) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kSliceWaves; ++w) v += part[(w * kOut + o) * 64 + lane];
    const int e = o & 3, s = (o >> 2) % NS, m = (o >> 2) / NS;
    const int64_t row = m0 + m * 16 + (lane >> 4) * 4 + e, n = n0 + s * 16 + (lane & 15);
    if (row < a.M && n < a.N) store_as(a.out, a.odt, (size_t)row * a.N + n, v);
  }
}

// (few slices: tile_launch)
template <class S, int FMT, int RAGGED, int MT, int NS>
hipError_t slice_launch(const RowsArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.N + NS * 16 - 1) / (NS * 16)), (unsigned)((a.M + MT * 16 - 1) / (MT * 16)));
  const size_t stage = (size_t)kSliceWaves * MT * 16 * 256, sums = (size_t)kSliceWaves * MT * NS * 1024;
  hipLaunchKernelGGL((q4_slice_kernel<S, FMT, RAGGED, MT, NS>), grid, dim3(64 * kSliceWaves),
                     stage > sums ? stage : sums, s, a);
  return hipGetLastError();
}

template <class S, int FMT, int RAGGED>
hipError_t whole_tiles(const RowsArgs& a, int64_t tn, int ncu, hipStream_t s) {
  for (int64_t row = 0; row < a.M;) {
    const TileLaunch t = tile_launch_at(row, a.M, tn, ncu);
    RowsArgs b = a;
    b.x = (const char*)a.x + (size_t)row * a.K * 2;
    b.out = (char*)a.out + (size_t)row * a.N * (a.odt == MOE_F32 ? 4 : 2);
    b.M = t.rows;
    hipLaunchKernelGGL((q4_tile_kernel<S, FMT, RAGGED>), dim3(t.grid), dim3(kTileThreads), 2 * kStage, s, b, (int)tn,
                       t.whole, t.tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    row += t.rows;
  }
  return hipSuccess;
}

template <class S, int FMT, int RAGGED>
hipError_t tile_launch(const RowsArgs& a, int ncu, hipStream_t s) {
  const int64_t tn = ((int64_t)a.N + kTileN - 1) / kTileN;
  const int64_t strips = ((int64_t)a.N + 15) / 16;
  // Slices of 64 x 64 against tiles, us at N = K = 4096: 300 rows 46 / 71, 640 rows 70 / 73,
  // 768 rows 71 / 73, 1024 rows 94 / 74, 2048 rows 183 / 114; at K = 14336 640 rows 196 / 230,
  // 1024 rows 292 / 243; at K = 1024, where a tile's start and end count less, 300 rows 20 / 25,
  // 640 rows 30 / 26. 33 rows of N = 32768 51 / 69, of 65536 101 / 75 (32 x 16: 17 rows 87 / 73).
  if ((a.M + 63) / 64 * (((int64_t)a.N + 63) / 64) > 3 * ncu) return whole_tiles<S, FMT, RAGGED>(a, tn, ncu, s);
  // 32 x 16 against 64 x 16 and 64 x 64 at 32 rows, K = 4096: N = 4096 9 / 12 / 22, 14336 24 / 46
  // / 26, 32768 43 / 85 / 50
  if (a.M <= 32) return slice_launch<S, FMT, RAGGED, 2, 1>(a, s);
  // 64 x 16 in one round, against 64 x 64: 64 rows of 4096 13 / 24 (K = 14336 50 / 72), 186 rows
  // of 1024 14 / 24; in more, 100 rows of 4096 28 / 25 (K = 14336 92 / 66), 300 of 1024 29 / 25
  const int64_t r64 = (a.M + 63) / 64;
  if (r64 * strips <= ncu) return slice_launch<S, FMT, RAGGED, 4, 1>(a, s);
  return slice_launch<S, FMT, RAGGED, 4, 4>(a, s);
}

template <class S>
hipError_t tile_format(const RowsArgs& a, int ncu, hipStream_t s) {
  switch (a.fmt) {
    case 0: return a.K % 64 ? tile_launch<S, 0, kOdd>(a, ncu, s) : tile_launch<S, 0, kWords>(a, ncu, s);
    case 1: return tile_launch<S, 1, kWords>(a, ncu, s);
    case 2: return tile_launch<S, 2, kWords>(a, ncu, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_q4_tile(const RowsArgs& a, int ncu, hipStream_t s) {
  return a.xdt == MOE_F16 ? tile_format<_Float16>(a, ncu, s) : tile_format<__bf16>(a, ncu, s);
}

}  // namespace moe
