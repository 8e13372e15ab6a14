// Products on 8-bit blocks, many rows: a 256 x 256 tile on gfx950.
//
// One block of 8 waves computes 256 weight rows x up to 256 rows; a wave
// owns 128 weight rows x 64, 32 or 16 rows (4, 2 or 1 fragments of 16: the
// tile's rows rounded up to 256, 128 or 64). K streams in steps of one scale
// block, 128 codes, through two LDS stages of 64 KB that buffer_load ... lds
// fills directly while the other is multiplied. A fragment's block sum
// starts from zero in the matrix unit and one fma a value adds it, scaled,
// to the f32 accumulators; these must lie in registers that vector
// instructions reach, which is what limits a wave to 128 x 64.
//
// PREC 0 multiplies the codes in the 8-bit matrix unit (16x16x128), at twice
// the rate of the 16-bit one. It aligns the products it adds to the largest
// and drops what lies 2^-14 below it, an error of 1.5e-5 of an output on
// normally distributed rows: for 16-bit outputs (half a step is 2^-9 or
// 2^-12 of the value) far less than their own rounding. PREC 1 widens the
// codes to f16 (exactly) and sums them in f32 throughout, for f32 outputs.
#include <algorithm>

#include "f8_common.h"

namespace moe {

namespace {

constexpr int kTW = 256;                 // weight rows of a tile
constexpr int kTT = 256;                 // rows of a tile
constexpr int kStageW = kTW * 128;       // bytes of a stage's weight codes
constexpr int kStageB = kStageW + kTT * 128;
constexpr int kScaleK = 32;              // blocks of K whose row scales are held at once
constexpr int kTileLds = 2 * kStageB + kScaleK * kTT * 4;   // 160 KB

// Fragments are read as vector types: a read of a struct (uint4) loses its
// type on the way to the instruction, and the compiler then guards it with a
// wait for every direct-to-LDS load in flight.
typedef int v4i32 __attribute__((ext_vector_type(4)));

// 16-byte piece c of row r of a stage lies at piece c ^ ((r >> 1) & 7) of
// the row's 128 bytes: the 16 rows that one fragment read touches then
// spread over all 64 banks.
__device__ __forceinline__ int piece(int r, int c) {
  return r * 128 + ((c ^ ((r >> 1) & 7)) << 4);
}

__device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }

}  // namespace

template <int MODE, int PREC>
__global__ __launch_bounds__(512, 1) void f8_tile_kernel(F8Args a) {
  __shared__ __attribute__((aligned(1024))) char smem[kTileLds];
  float* const srow = reinterpret_cast<float*>(smem + 2 * kStageB);   // [kScaleK][kTT]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ww = wave >> 2, wt = wave & 3;
  const int lr = lane & 15, lq = lane >> 4;
  const int K = a.K, N = a.N;
  const int nk = (K + 127) / 128;
  const int NNB = MODE == 1 ? N / 128 : (N + kTW - 1) / kTW;
  const int n_tiles = MODE == 0 ? (int)((a.M + kTT - 1) / kTT) : a.meta[a.meta_index];
  const int n_items = n_tiles * NNB;
  const int b = xcd_item(0, blockIdx.x, gridDim.x, n_items);
  if (b < 0) return;   // the whole block, before any barrier
  // 4 row tiles x all column blocks at a time, rows first
  const int group = b / (4 * NNB), first = group * 4;
  const int gm = min(4, n_tiles - first);
  const int within = b - first * NNB;
  const int ti = first + within % gm, nb = within / gm;
  int e = 0, rows;
  int64_t row0;
  if (MODE == 0) {
    row0 = (int64_t)ti * kTT;
    rows = (int)min((int64_t)kTT, a.M - row0);
  } else {
    e = a.list[2 * ti];
    const int r0 = a.list[2 * ti + 1], off = a.offsets[e];
    row0 = off + r0;
    rows = min(kTT, a.offsets[e + 1] - off - r0);
  }
  const int n0 = nb * (MODE == 1 ? 128 : kTW);

  auto run = [&](auto tb_c) {
    constexpr int TB = decltype(tb_c)::value;   // 16-row fragments a wave
    // ---- this lane's sources of a stage: wave w fills weight rows 32 w ..
    // 32 w + 31 (four loads of 8 rows) and rows 8 TB w .. of the tile
    const int dr = lane >> 3, dc = lane & 7;
    const size_t mat = (size_t)e * N * K;
    const __amdgpu_buffer_rsrc_t rw0 =
        make_rsrc(a.B0 + mat + (size_t)n0 * K, (uint32_t)(min(kTW, N - n0) * (int64_t)K));
    const __amdgpu_buffer_rsrc_t rw1 =
        MODE == 1 ? make_rsrc(a.B1 + mat + (size_t)n0 * K, (uint32_t)(128 * (int64_t)K)) : rw0;
    const __amdgpu_buffer_rsrc_t rt =
        MODE == 1 ? make_rsrc(a.A, 0x7FFFFFFFu)
                  : make_rsrc(a.A + (size_t)row0 * K, (uint32_t)(rows * (int64_t)K));
    uint32_t vw[4], vt[TB];
    int cw[4], ct[TB];   // byte of the row at which the lane's piece starts
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int R = 32 * wave + 8 * j + dr;
      cw[j] = (dc ^ ((R >> 1) & 7)) * 16;
      int row = R;
      // gate/up: fragments of 16 rows alternate W_gate / W_up, 64 features
      // a half of the tile
      if (MODE == 1) row = (R >> 7) * 64 + ((R >> 5) & 3) * 16 + (R & 15);
      else row = min(R, N - n0 - 1);
      vw[j] = (uint32_t)row * (uint32_t)K + (uint32_t)cw[j];
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const int R = (wave * TB + j) * 8 + dr;
      ct[j] = (dc ^ ((R >> 1) & 7)) * 16;
      const int rr = min(R, rows - 1);
      const int src = MODE == 1 ? a.pair_token[row0 + rr] : rr;
      vt[j] = (uint32_t)src * (uint32_t)K + (uint32_t)ct[j];
    }
    auto issue = [&](int kt) {
      char* st = smem + (kt & 1) * kStageB;
      const int k0 = kt * 128;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // gate/up: rows 16..31 of every 32 are W_up's
        const __amdgpu_buffer_rsrc_t r = MODE == 1 && (j & 2) ? rw1 : rw0;
        uint32_t v = vw[j];
        if (MODE == 0 && k0 + cw[j] >= K) v = 0x80000000u;   // past the row: zeros
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(st + (wave * 4 + j) * 1024), 16,
                                                 (int)v, k0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        uint32_t v = vt[j];
        if (MODE == 0 && k0 + ct[j] >= K) v = 0x80000000u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rt, (lds_ptr_t)(st + kStageW + (wave * TB + j) * 1024), 16, (int)v, k0, 0, 0);
      }
    };
    // row scales of blocks kc .. kc + kScaleK - 1 to srow[block][row]: lane
    // groups of 16 take neighbouring blocks of one row
    auto load_scales = [&](int kc) {
      const int nc = min(kScaleK, nk - kc);
      for (int i = tid; i < 64 * TB * 16; i += 512) {
        const int r = i >> 4;
        const int rr = min(r, rows - 1);
        const int64_t src = MODE == 1 ? (int64_t)a.pair_token[row0 + rr] : row0 + rr;
        for (int c = i & 15; c < nc; c += 16) srow[c * kTT + r] = a.As[src * nk + kc + c];
      }
    };
    // the weights' scales: one a wave's 128 rows and block (gate/up: one of
    // each matrix)
    const int nn = (N + 127) / 128;
    const int sb = MODE == 1 ? nb : min(nb * 2 + ww, nn - 1);
    const float* ws0 = a.B0s + ((size_t)e * nn + sb) * nk;
    const float* ws1 = MODE == 1 ? a.B1s + ((size_t)e * nn + sb) * nk : ws0;

    floatx4 acc[8][TB];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int t = 0; t < TB; ++t) acc[i][t] = floatx4{0.f, 0.f, 0.f, 0.f};

    using Frag = std::conditional_t<PREC == 0, v8i32, Codes>;
    auto frag = [&](const char* base, int r) {
      const v4i32 lo = *reinterpret_cast<const v4i32*>(base + piece(r, 2 * lq));
      const v4i32 hi = *reinterpret_cast<const v4i32*>(base + piece(r, 2 * lq + 1));
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
    // the weights' scales of the held blocks, one a lane (a load inside the
    // K loop would wait for every load of the next stage)
    float wl0 = 0.f, wl1 = 0.f;
    auto lane_of = [](float v, int l) {
      return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
    };

    issue(0);
    for (int kt = 0; kt < nk; ++kt) {
      const int kc = kt % kScaleK;
      if (kc == 0) {
        // the previous scales' readers are past this barrier
        if (kt) { fence(); __builtin_amdgcn_s_barrier(); fence(); }
        load_scales(kt);
        const int c = min(kt + (lane & (kScaleK - 1)), nk - 1);
        wl0 = ws0[c];
        if (MODE == 1) wl1 = ws1[c];
      }
      // this wave's loads have landed (and its scale writes); after the
      // barrier every wave's have, and every wave is past its reads of the
      // other stage, which the next loads fill
      fence();
      wait_vm_lgkm0<0>();
      __builtin_amdgcn_s_barrier();
      fence();
      if (kt + 1 < nk) issue(kt + 1);
      const char* sw = smem + (kt & 1) * kStageB;
      const char* st = sw + kStageW;
      Frag xt[TB], wv;
      v8i32 wf[2];
      float s0[TB], s1[TB];
      const float w0 = lane_of(wl0, kc), w1 = MODE == 1 ? lane_of(wl1, kc) : w0;
      wf[0] = frag(sw, ww * 128 + lr);
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const int r = (wt * TB + t) * 16 + lr;
        xt[t] = operand(frag(st, r));
        const float sr = srow[kc * kTT + r];
        s0[t] = sr * w0;
        s1[t] = MODE == 1 ? sr * w1 : s0[t];
      }
      // block sums go to the accumulators kLag products later, so that a
      // wave's matrix instructions do not wait for one another's results
      constexpr int kN = 8 * TB, kLag = PREC == 0 ? 2 : 1;
      floatx4 p[kLag + 1];
#pragma unroll
      for (int j = 0; j < kN + kLag; ++j) {
        if (j < kN) {
          const int i = j / TB, t = j % TB;
          if (t == 0) {
            wv = operand(wf[i & 1]);
            if (i < 7) wf[(i + 1) & 1] = frag(sw, ww * 128 + (i + 1) * 16 + lr);
          }
          p[j % (kLag + 1)] = product(wv, xt[t]);
        }
        if (j >= kLag) {
          const int d = j - kLag, i = d / TB, t = d % TB;
          const float sc = (i & 1) ? s1[t] : s0[t];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[i][t][q] = fmaf(p[d % (kLag + 1)][q], sc, acc[i][t][q]);
        }
      }
    }

    // ---- epilogue
    if constexpr (MODE == 1) {
      // h of 64 features a wave; a block's largest magnitude is the maximum
      // over the lane's four groups, the four lane groups and both halves
      fence();
      __builtin_amdgcn_s_barrier();   // every wave is done with the stages
      fence();
      uint32_t* mx = reinterpret_cast<uint32_t*>(smem);   // [2][kTT]
      uint32_t m[TB];
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        m[t] = 0;
#pragma unroll
        for (int i = 0; i < 8; i += 2)
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
        const F8Scale sc = f8_scale(max(mx[r], mx[kTT + r]));
        const size_t pr = (size_t)(row0 + r);
        if (ww == 0 && lq == 0) a.out_s[pr * (N / 128) + nb] = sc.s;
        uint8_t* dst = static_cast<uint8_t*>(a.out) + pr * N + n0 + ww * 64 + lq * 4;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          int w = 0;
          w = __builtin_amdgcn_cvt_pk_fp8_f32(acc[i][t][0] * sc.inv, acc[i][t][1] * sc.inv, w, false);
          w = __builtin_amdgcn_cvt_pk_fp8_f32(acc[i][t][2] * sc.inv, acc[i][t][3] * sc.inv, w, true);
          *reinterpret_cast<int*>(dst + i * 8) = w;
        }
      }
    } else {
      const bool vec = (N & 3) == 0;
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const int r = (wt * TB + t) * 16 + lr;
        if (r >= rows) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int n = n0 + ww * 128 + i * 16 + lq * 4;
          const size_t at = (size_t)(row0 + r) * N + n;
          const float v[4] = {acc[i][t][0], acc[i][t][1], acc[i][t][2], acc[i][t][3]};
          if (vec) {
            if (n < N) store_out4(a.out, a.odt, at, v);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (n + q < N) store_out1(a.out, a.odt, at + q, v[q]);
          }
        }
      }
    }
  };
  if (rows > 128) run(std::integral_constant<int, 4>{});
  else if (rows > 64) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 1>{});
}

hipError_t launch_f8_tile(const F8Args& a, int prec, hipStream_t s) {
  const int64_t tiles = a.mode == 0 ? (a.M + kTT - 1) / kTT : a.max_groups;
  const int64_t items = tiles * (a.mode == 1 ? a.N / 128 : (a.N + kTW - 1) / kTW);
  if (items == 0) return hipSuccess;
  const dim3 grid((unsigned)((items + 7) / 8 * 8)), block(512);
  if (prec) {
    if (a.mode == 0) hipLaunchKernelGGL((f8_tile_kernel<0, 1>), grid, block, 0, s, a);
    else if (a.mode == 1) hipLaunchKernelGGL((f8_tile_kernel<1, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((f8_tile_kernel<2, 1>), grid, block, 0, s, a);
  } else {
    if (a.mode == 0) hipLaunchKernelGGL((f8_tile_kernel<0, 0>), grid, block, 0, s, a);
    else if (a.mode == 1) hipLaunchKernelGGL((f8_tile_kernel<1, 0>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((f8_tile_kernel<2, 0>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
