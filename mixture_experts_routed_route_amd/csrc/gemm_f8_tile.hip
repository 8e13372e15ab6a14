// Products on 8-bit blocks, many rows: a 256 x 256 tile on gfx950.
//
// One block of 8 waves computes 256 weight rows x up to 256, 128 or 64 rows;
// the waves stand 2 x 4, 4 x 2 or 8 x 1, so that each owns 64 rows and 128,
// 64 or 32 weight rows (the layout that reads the fewest fragments from LDS
// at each size). K streams in steps of one scale
// block, 128 codes, through two LDS stages of 64 KB that buffer_load ... lds
// fills directly while the other is multiplied. A fragment's block sum
// starts from zero in the matrix unit and one fma a value adds it, scaled,
// to the f32 accumulators; these must lie in registers that vector
// instructions reach, which is what limits a wave to 128 x 64.
//
// PREC 0 multiplies the codes in the 8-bit matrix unit (16x16x128), at twice
// the rate of the 16-bit one. It aligns the products it adds to the largest
// and drops what lies 2^-13 below it, an error of 1.5e-5 of an output on
// normally distributed rows: for 16-bit outputs (half a step is up to 2^-8 or
// 2^-11 of the value) far less than their own rounding. PREC 1 widens the
// codes to f16 (exactly) and sums them in f32 throughout, for f32 outputs (a
// layer's down products where y is f32) and for gate/up: h is coded next, and the few codes that an error of its sums
// moves over a border move by a whole step. With PREC 0 there a bf16 layer of
// 4096 tokens was 2.0e-3 from the exact y, not 1.7e-3.
//
// 13312 x 4096 x 4096 to f16: 225 us, 1.99 PFLOP/s; to f32 390 us, 1.14. A
// library product of the same codes with one scale for a whole tensor takes 202
// to 231. Traced, the matrix units are busy for 46 % of the cycles at 2.11 GHz
// (zeros: 47 % at 2.32; to f32 48 % at 2.31; the library's 49 % at 2.14), so
// power takes a tenth of the clock, and over half of the cycles go to the 128
// fma a lane and step that scale and add the blocks' sums, which both waves of a
// SIMD do at the same time, to the barrier of a step, and to a tile's ends.
#include <algorithm>

#include "f8_common.h"

namespace moe {

namespace {

constexpr int kTW = 256;                 // weight rows of a tile
constexpr int kTT = 256;                 // rows of a tile
constexpr int kStageW = kTW * 128;       // bytes of a stage's weight codes
constexpr int kStageB = kStageW + kTT * 128;
constexpr int kScaleK = 4;               // blocks of K whose row scales are loaded at once
constexpr int kTileLds = 2 * kStageB + 2 * kScaleK * kTT * 4;   // 136 KB

// Fragments are read as vector types: a read of a struct (uint4) loses its
// type on the way to the instruction, and the compiler then guards it with a
// wait for every direct-to-LDS load in flight.
typedef int v4i32 __attribute__((ext_vector_type(4)));

// 16-byte piece c of row r of a stage lies at piece c ^ ((r >> 1) & 7) of
// the row's 128 bytes. Lane group q of a fragment reads pieces q and q + 4
// (both operands the same, so the order of K within a block is free): the
// LDS serves a 16-byte read in groups of 16 lanes such as 0-3, 12-15, 20-27,
// and these then touch all 64 banks once (pieces 2 q and 2 q + 1 met in
// pairs: half of the LDS cycles of an 8192^3 product were conflicts).
__device__ __forceinline__ int piece(int r, int c) {
  return r * 128 + ((c ^ ((r >> 1) & 7)) << 4);
}

__device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }

}  // namespace

template <int MODE, int PREC>
__global__ __launch_bounds__(512, 1) void f8_tile_kernel(F8Args a) {
  __shared__ __attribute__((aligned(1024))) char smem[kTileLds];
  float* const srow = reinterpret_cast<float*>(smem + 2 * kStageB);   // [2 kScaleK][kTT]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int K = a.K, N = a.N;
  const int nk = (K + 127) / 128;
  const int NNB = MODE == 1 ? N / 128 : (N - 1) / kTW + 1;
  // Block b runs on XCD b mod 8, whose L2 its neighbours share.
  int ti, nb;
  if (MODE == 0) {
    // a.tiles256 tiles of 256 rows, then tiles of a.tail_rows; each kind's
    // items in eight contiguous runs, one an XCD, four row tiles by all
    // column blocks at a time
    const int n_big = a.tiles256 * NNB, g_big = (n_big + 7) & ~7;
    const bool big = (int)blockIdx.x < g_big;
    const int n = big ? a.tiles256 : a.tail_tiles;
    const int it = big ? xcd_item(0, blockIdx.x, g_big, n_big)
                       : xcd_item(0, blockIdx.x - g_big, gridDim.x - g_big, n * NNB);
    if (it < 0) return;   // the whole block, before any barrier
    const int first = it / (4 * NNB) * 4;
    const int gm = min(4, n - first), within = it - first * NNB;
    ti = first + within % gm + (big ? 0 : a.tiles256);
    nb = within / gm;
  } else {
    // the list's tiles, most rows first, go to the XCDs in turn
    const int m = blockIdx.x >> 3;
    ti = m / NNB * 8 + (blockIdx.x & 7);
    nb = m % NNB;
    if (ti >= *a.groups) return;
  }
  int e = 0, rows;
  int64_t row0;
  if (MODE == 0) {
    const int tail = ti - a.tiles256;
    row0 = tail < 0 ? (int64_t)ti * kTT
                    : (int64_t)a.tiles256 * kTT + (int64_t)tail * a.tail_rows;
    rows = (int)min((int64_t)(tail < 0 ? kTT : a.tail_rows), a.M - row0);
  } else {
    e = a.list[2 * ti];
    const int r0 = a.list[2 * ti + 1], off = a.offsets[e];
    row0 = off + r0;
    rows = min(kTT, a.offsets[e + 1] - off - r0);
  }
  const int n0 = nb * (MODE == 1 ? 128 : kTW);

  // NW waves along the weight rows, 8 / NW along the rows
  auto run = [&](auto nw_c) {
    constexpr int NW = decltype(nw_c)::value, NT = 8 / NW;
    constexpr int FW = 16 / NW;      // a wave's fragments of 16 weight rows
    constexpr int TB = 4;            // and of 16 rows
    constexpr int DT = NT;           // 8-row loads of a wave's share of a stage's rows
    const int ww = wave / NT, wt = wave % NT;
    // ---- this lane's sources of a stage: wave w fills weight rows 32 w ..
    // 32 w + 31 (four loads of 8 rows) and rows 8 DT w .. of the tile
    const int dr = lane >> 3, dc = lane & 7;
    const size_t mat = (size_t)e * N * K;
    const __amdgpu_buffer_rsrc_t rw0 =
        make_rsrc(a.B0 + mat + (size_t)n0 * K, (uint32_t)(min(kTW, N - n0) * (int64_t)K));
    const __amdgpu_buffer_rsrc_t rw1 =
        MODE == 1 ? make_rsrc(a.B1 + mat + (size_t)n0 * K, (uint32_t)(128 * (int64_t)K)) : rw0;
    const __amdgpu_buffer_rsrc_t rt =
        MODE == 1 ? make_rsrc(a.A, 0x7FFFFFFFu)
                  : make_rsrc(a.A + (size_t)row0 * K, (uint32_t)(rows * (int64_t)K));
    uint32_t vw[4], vt[DT];
    // byte of the row at which the lane's piece starts, for even and odd
    // groups of 8 stage rows
    const int cb[2] = {(dc ^ (dr >> 1)) * 16, (dc ^ (dr >> 1) ^ 4) * 16};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int R = 32 * wave + 8 * j + dr;
      int row = R;
      // gate/up: fragments of 16 rows alternate W_gate / W_up
      if (MODE == 1) row = (R >> 5) * 16 + (R & 15);
      else row = min(R, N - n0 - 1);
      vw[j] = (uint32_t)row * (uint32_t)K + (uint32_t)cb[j & 1];
    }
#pragma unroll
    for (int j = 0; j < DT; ++j) {
      const int R = (wave * DT + j) * 8 + dr;
      const int rr = min(R, rows - 1);
      const int src = MODE == 1 ? a.pair_token[row0 + rr] : rr;
      vt[j] = (uint32_t)src * (uint32_t)K + (uint32_t)cb[(DT == 1 ? wave : j) & 1];
    }
    auto issue = [&](int kt) {
      char* st = smem + (kt & 1) * kStageB;
      const int k0 = kt * 128;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // gate/up: rows 16..31 of every 32 are W_up's
        const __amdgpu_buffer_rsrc_t r = MODE == 1 && (j & 2) ? rw1 : rw0;
        uint32_t v = vw[j];
        if (MODE == 0 && k0 + cb[j & 1] >= K) v = 0x80000000u;   // past the row: zeros
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(st + (wave * 4 + j) * 1024), 16,
                                                 (int)v, k0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < DT; ++j) {
        uint32_t v = vt[j];
        if (MODE == 0 && k0 + cb[(DT == 1 ? wave : j) & 1] >= K) v = 0x80000000u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rt, (lds_ptr_t)(st + kStageW + (wave * DT + j) * 1024), 16, (int)v, k0, 0, 0);
      }
    };
    // Row scales, four blocks at a time: thread (row, half) loads two of them
    // with the first stage of the four before, and writes them to LDS one
    // step later, when every load has landed anyway.
    const int sc_r = tid & (kTT - 1), sc_h = 2 * (tid >> 8);
    const __amdgpu_buffer_rsrc_t rs =
        make_rsrc(MODE == 1 ? a.As : a.As + (size_t)row0 * nk, 0x7FFFFFFFu);
    uint32_t sc_off;
    {
      const int rr = min(sc_r, rows - 1);
      sc_off = (uint32_t)(MODE == 1 ? a.pair_token[row0 + rr] : rr) * (uint32_t)nk * 4u;
    }
    float sc_v[2];
    auto load_scales = [&](int kb) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        sc_v[j] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            rs, (int)(sc_off + (uint32_t)min(kb + sc_h + j, nk - 1) * 4u), 0, 0));
    };
    auto write_scales = [&](int kb) {
#pragma unroll
      for (int j = 0; j < 2; ++j) srow[((kb & 4) + sc_h + j) * kTT + sc_r] = sc_v[j];
    };
    // the weights' scales: one a wave's 128 rows and block (gate/up: one of
    // each matrix)
    const int nn = (N - 1) / 128 + 1;
    const int sb = MODE == 1 ? nb : min(nb * 2 + ww / (NW / 2), nn - 1);
    const float* ws0 = a.B0s + ((size_t)e * nn + sb) * nk;
    const float* ws1 = MODE == 1 ? a.B1s + ((size_t)e * nn + sb) * nk : ws0;

    using Frag = std::conditional_t<PREC == 0, v8i32, Codes>;
    auto frag = [&](const char* base, int r) {
      const v4i32 lo = *reinterpret_cast<const v4i32*>(base + piece(r, lq));
      const v4i32 hi = *reinterpret_cast<const v4i32*>(base + piece(r, lq + 4));
      return (v8i32)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto operand = [&](const v8i32& v) -> Frag {
      if constexpr (PREC == 0) return v;
      else return widen(v);
    };
    auto product = [&](const Frag& x, const Frag& y) {
      if constexpr (PREC == 0) return mfma_f8(x, y, floatx4{0.f, 0.f, 0.f, 0.f});
      else return block_product(x, y);
    };
    // the weights' scales of 64 blocks, one a lane (a load at every step
    // would wait for every load of the next stage)
    float wl0 = 0.f, wl1 = 0.f;
    auto lane_of = [](float v, int l) {
      return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
    };

    auto fill_weights = [&](int kb) {
      const int c = min(kb + lane, nk - 1);
      wl0 = ws0[c];
      if (MODE == 1) wl1 = ws1[c];
    };
    fill_weights(0);
    load_scales(0);
    issue(0);
    write_scales(0);
    floatx4 acc[FW][TB];
#pragma unroll
    for (int i = 0; i < FW; ++i)
#pragma unroll
      for (int t = 0; t < TB; ++t) acc[i][t] = floatx4{0.f, 0.f, 0.f, 0.f};

    // Once every wave is past its reads of stage kn - 1 and its loads of
    // stage kn (and its scale writes) have landed: the next stage's loads and
    // the scales of the blocks ahead.
    auto next_stage = [&](int kn) {
      fence();
      wait_vm_lgkm0<0>();
      __builtin_amdgcn_s_barrier();
      fence();
      if ((kn & 3) == 1 && kn + 3 < nk) write_scales(kn + 3);
      if (kn && (kn & 63) == 0) {
        fill_weights(kn);
        // waited for here, before the next stage's loads: at their use the
        // wait would cover those too
        wait_vmcnt<0>();
        asm volatile("" : "+v"(wl0), "+v"(wl1));
      }
      if ((kn & 3) == 0 && kn + 4 < nk) load_scales(kn + 4);
      if (kn + 1 < nk) issue(kn + 1);
    };
    auto row_scale = [&](int kt, int t) {
      return srow[(kt & 7) * kTT + (wt * TB + t) * 16 + lr];
    };
    Frag xt[TB], wv;
    v8i32 wf[2];
    float sr[TB], s0[TB], s1[TB];
    auto first_weights = [&](int kt) {
      wf[0] = frag(smem + (kt & 1) * kStageB, ww * FW * 16 + lr);
    };
    auto row_fragment = [&](int kt, int t) {
      xt[t] = operand(frag(smem + (kt & 1) * kStageB + kStageW, (wt * TB + t) * 16 + lr));
      sr[t] = row_scale(kt, t);
    };
    next_stage(0);
    first_weights(0);
#pragma unroll
    for (int t = 0; t < TB; ++t) row_fragment(0, t);
    for (int kt = 0; kt < nk; ++kt) {
      const char* sw = smem + (kt & 1) * kStageB;
      const float w0 = lane_of(wl0, kt & 63), w1 = MODE == 1 ? lane_of(wl1, kt & 63) : w0;
      // Block sums go to the accumulators kLag products later, so that a
      // wave's matrix instructions do not wait for one another's results.
      // The stages change hands before the last weight fragment's products,
      // whose rows' registers then take the next step's fragments one by
      // one: the next step's products start without a wait.
      constexpr int kN = FW * TB, kLag = PREC == 0 ? 3 : 1;
      floatx4 p[kLag + 1];
#pragma unroll
      for (int j = 0; j < kN + kLag; ++j) {
        if (j < kN) {
          const int i = j / TB, t = j % TB;
          if (t == 0) {
            wv = operand(wf[i & 1]);
            if (i < FW - 1) {
              wf[(i + 1) & 1] = frag(sw, (ww * FW + i + 1) * 16 + lr);
            } else {   // after the last step: a barrier, and reads of no use
              next_stage(kt + 1);
              if (PREC == 0) first_weights(kt + 1);
            }
          }
          p[j % (kLag + 1)] = product(wv, xt[t]);
          if (PREC == 0 && i == FW - 1) row_fragment(kt + 1, t);
        }
        // the step's scales, one by one before the first sums that take them
        // (all at once would wait for the last row's reads)
        if (j >= kLag - 1 && j < kLag - 1 + TB) {
          const int t = j - (kLag - 1);
          s0[t] = sr[t] * w0;
          s1[t] = MODE == 1 ? sr[t] * w1 : s0[t];
        }
        if (j >= kLag) {
          const int d = j - kLag, i = d / TB, t = d % TB;
          const float sc = (i & 1) ? s1[t] : s0[t];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[i][t][q] = fmaf(p[d % (kLag + 1)][q], sc, acc[i][t][q]);
          // here, not behind the branches of next_stage
          asm volatile("" : "+v"(acc[i][t]));
        }
        // keeps this order: the scheduler would bring each sum back next to
        // its product and fill the wait with no-ops
        if (PREC == 0) __builtin_amdgcn_sched_barrier(0);
      }
      if (PREC != 0) {   // widened rows: no registers to spare
        first_weights(kt + 1);
#pragma unroll
        for (int t = 0; t < TB; ++t) row_fragment(kt + 1, t);
      }
    }

    // ---- epilogue
    if constexpr (MODE == 1) {
      // h of 128 / NW features a wave; a block's largest magnitude is the
      // maximum over a lane's, the four lane groups' and the NW waves' values
      fence();
      __builtin_amdgcn_s_barrier();   // every wave is done with the stages
      fence();
      uint32_t* mx = reinterpret_cast<uint32_t*>(smem);   // [NW][kTT]
      uint32_t m[TB];
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        m[t] = 0;
#pragma unroll
        for (int i = 0; i < FW; i += 2)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float h = swiglu(acc[i][t][q], acc[i + 1][t][q], a.clamp);
            acc[i][t][q] = h;
            m[t] = max(m[t], mag_bits(h));
          }
        m[t] = max(m[t], (uint32_t)__shfl_xor((int)m[t], 16));
        m[t] = max(m[t], (uint32_t)__shfl_xor((int)m[t], 32));
        if (lq == 0) mx[ww * kTT + (wt * TB + t) * 16 + lr] = m[t];
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const int r = (wt * TB + t) * 16 + lr;
        if (r >= rows) continue;
        uint32_t mm = mx[r];
#pragma unroll
        for (int w = 1; w < NW; ++w) mm = max(mm, mx[w * kTT + r]);
        const F8Scale sc = f8_scale(mm);
        const size_t pr = (size_t)(row0 + r);
        if (ww == 0 && lq == 0) a.out_s[pr * (N / 128) + nb] = sc.s;
        uint8_t* dst = static_cast<uint8_t*>(a.out) + pr * N + n0 + ww * FW * 8 + lq * 4;
#pragma unroll
        for (int i = 0; i < FW; i += 2) {
          int w = 0;
          w = __builtin_amdgcn_cvt_pk_fp8_f32(acc[i][t][0] * sc.inv, acc[i][t][1] * sc.inv, w, false);
          w = __builtin_amdgcn_cvt_pk_fp8_f32(acc[i][t][2] * sc.inv, acc[i][t][3] * sc.inv, w, true);
          *reinterpret_cast<int*>(dst + i * 8) = w;
        }
      }
    } else {
      if ((N & (a.odt == MOE_F32 ? 3 : 7)) == 0) {   // 16-byte stores
        // Through LDS, 128 rows at a time, so that a store covers whole rows of
        // the tile. Lanes hold four columns of 16 rows; stored from there, 64
        // or 32 bytes a row, a bf16 product of 4096^3 took 68 us, not 65, and
        // a 4096-token layer's down product (K = 768, f32) 128 us, not 119.
        // Piece c (four columns) of row r lies at piece c ^ (r & 15).
        float* const tile = reinterpret_cast<float*>(smem);   // [128][kTW]
        auto at = [](int r, int c) { return r * kTW + ((c ^ (r & 15)) << 2); };
#pragma unroll
        for (int h = 0; h < (NT > 2 ? 2 : 1); ++h) {
          fence();
          wait_vm_lgkm0<63>();
          __builtin_amdgcn_s_barrier();   // the stages, or the half before, have been read
          fence();
          if (NT <= 2 || wt >> 1 == h) {
#pragma unroll
            for (int t = 0; t < TB; ++t)
#pragma unroll
              for (int i = 0; i < FW; ++i)
                *reinterpret_cast<floatx4*>(
                    tile + at((wt * TB + t) * 16 + lr - 128 * h, (ww * FW + i) * 4 + lq)) = acc[i][t];
          }
          fence();
          wait_vm_lgkm0<63>();
          __builtin_amdgcn_s_barrier();
          fence();
          const int rh = min(128, rows - 128 * h);
          const size_t r0 = (size_t)(row0 + 128 * h);
          if (a.odt == MOE_F32) {
#pragma unroll 4
            for (int r = wave; r < rh; r += 8) {
              const floatx4 v = *reinterpret_cast<const floatx4*>(tile + at(r, lane));
              if (n0 + lane * 4 < N)
                *reinterpret_cast<floatx4*>(static_cast<float*>(a.out) + (r0 + r) * N + n0 +
                                            lane * 4) = v;
            }
          } else {
            const int c = lane & 31;
#pragma unroll 4
            for (int r = wave * 2 + (lane >> 5); r < rh; r += 16) {
              const floatx4 x = *reinterpret_cast<const floatx4*>(tile + at(r, 2 * c));
              const floatx4 y = *reinterpret_cast<const floatx4*>(tile + at(r, 2 * c + 1));
              const float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
              if (n0 + c * 8 < N) store8(a.out, a.odt, (r0 + r) * N + n0 + c * 8, v);
            }
          }
        }
      } else {
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          const int r = (wt * TB + t) * 16 + lr;
          if (r >= rows) continue;
#pragma unroll
          for (int i = 0; i < FW; ++i) {
            const int n = n0 + (ww * FW + i) * 16 + lq * 4;
            const size_t at = (size_t)(row0 + r) * N + n;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (n + q < N) store_out1(a.out, a.odt, at + q, acc[i][t][q]);
          }
        }
      }
    }
  };
  if (rows > 128) run(std::integral_constant<int, 2>{});
  else if (rows > 64) run(std::integral_constant<int, 4>{});
  else run(std::integral_constant<int, 8>{});
}

hipError_t launch_f8_tile(const F8Args& a, int prec, hipStream_t s) {
  const int64_t tiles = a.mode == 0 ? a.tiles256 + a.tail_tiles : a.max_groups;
  const int64_t nnb = a.mode == 1 ? a.N / 128 : ((int64_t)a.N + kTW - 1) / kTW;
  if (tiles * nnb == 0) return hipSuccess;
  const int64_t blocks = a.mode == 0
      ? (a.tiles256 * nnb + 7) / 8 * 8 + (a.tail_tiles * nnb + 7) / 8 * 8
      : (tiles + 7) / 8 * 8 * nnb;
  const dim3 grid((unsigned)blocks), block(512);
  if (prec) {
    if (a.mode == 0) hipLaunchKernelGGL((f8_tile_kernel<0, 1>), grid, block, 0, s, a);
    else if (a.mode == 1) hipLaunchKernelGGL((f8_tile_kernel<1, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((f8_tile_kernel<2, 1>), grid, block, 0, s, a);
  } else {
    if (a.mode == 0) hipLaunchKernelGGL((f8_tile_kernel<0, 0>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((f8_tile_kernel<2, 0>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
