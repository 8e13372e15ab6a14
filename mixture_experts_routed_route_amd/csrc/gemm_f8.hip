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

// Strips: a wave takes 16 weight rows (gate/up: 16 of each matrix) against
// up to 16 RB rows of one group, weight operands straight from memory to
// registers (each weight code is used by one wave only). A workgroup of four
// waves takes 4 / ks strips, ks waves sharing one's blocks of K, their partial
// sums meeting in LDS: as many as leave each a block (from 16 blocks on only,
// 64 x 512 . 4096 x 512 took 9.1 us, not 5.9; from 64 on, 8 x 4096 . 1024 x
// 4096 12.1, not 7.9). A wave holds one block of loads at a time: in launches
// of many workgroups the up to eight of a CU cover one another's waits. One
// row of 2048 values by 4096 is 256 workgroups, one a CU, whose waves take four
// blocks in turn: 4.8 us (1.7 TB/s of weights), four waits that nothing covers.
//
// SRC 0 (plain products) reads quantised rows. SRC 1 (decode-shaped plans)
// reads the rows as they are (x in its type, or h in f32) and quantises the
// group's into LDS first, every workgroup for itself: for so few rows this
// costs less than a launch that quantises them once, and streams. us of a
// layer so / so: 2 tokens, top-8 of 128, D 2048, F 768 25 / 43, 8 tokens 61 /
// 64; 16 tokens, top-2 of 16, D 1536, F 256 21 / 31, top-4 at D 2048, F 768
// (34 KB of rows) 31 / 35.
constexpr int kStripLds = 49152;   // bytes of rows a workgroup may hold (SRC 1)

__host__ __device__ constexpr int strip_share(int nkb) { return nkb >= 4 ? 4 : nkb >= 2 ? 2 : 1; }

template <int MODE, int RB, int SRC>
__global__ __launch_bounds__(256) void f8_strip_kernel(F8Args a) {
  constexpr int WF = MODE == 1 ? 2 : 1;
  __shared__ float part[3][WF][RB][256];
  extern __shared__ __attribute__((aligned(16))) char rows_lds[];   // SRC 1
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int K = a.K, N = a.N;
  // N may be any size up to 2^31 - 1: no sum past it
  const int nkb = (K + 127) / 128, nnb = (N - 1) / 128 + 1;
  const int ks = strip_share(nkb), spw = 4 / ks;
  const int kw = wave & (ks - 1);          // this wave's share of K
  const int strips = (N - 1) / 16 + 1;
  const int sblocks = (strips + spw - 1) / spw;
  const int64_t groups = MODE == 0 ? (a.M + 16 * RB - 1) / (16 * RB) : *a.groups;
  const int64_t items = groups * sblocks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t gi = it / sblocks;
    // a strip past the last repeats it and stores nothing
    const int strip = (int)(it - gi * sblocks) * spw + wave / ks;
    const int n0 = min(strip, strips - 1) * 16;
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
      w[f] = (f ? a.B1 : a.B0) + ((size_t)e * N + n) * K + lq * 16;
      ws[f] = (f ? a.B1s : a.B0s) + ((size_t)e * nnb + (n0 >> 7)) * nkb;
    }
    v8i32 wv[WF];
    auto load_weights = [&](int kb) {
#pragma unroll
      for (int f = 0; f < WF; ++f) wv[f] = load_codes(w[f], lq, kb * 128, K);
    };
    load_weights(kw);
    const uint8_t* x[RB];
    const float* xs[RB];
    if constexpr (SRC == 0) {
#pragma unroll
      for (int t = 0; t < RB; ++t) {
        int64_t r = row0 + min(16 * t + lr, rows - 1);
        if (MODE == 1) r = a.pair_token[r];
        x[t] = a.A + (size_t)r * K + lq * 16;
        xs[t] = a.As + (size_t)r * nkb;
      }
    } else {
      // 16 lanes a block; rows 16 bytes apart beyond their codes, so that a
      // fragment's 16 rows lie on banks of their own
      const int nb = K / 128;
      float* const sl = reinterpret_cast<float*>(rows_lds + a.lds_rows * (K + 16));
      for (int i = threadIdx.x >> 4; i < rows * nb; i += 16) {
        const int r = i / nb, b = i - r * nb, k = b * 128 + (threadIdx.x & 15) * 8;
        const int64_t src = MODE == 1 ? (int64_t)a.pair_token[row0 + r] : row0 + r;
        float v[8];
        raw8_to_f32(load_raw8(a.A, a.adt, (size_t)src * K + k), a.adt, v);
        const F8Scale sc = f8_scale(max16(mag_max8(v)));
        *reinterpret_cast<uint2*>(rows_lds + r * (K + 16) + k) = f8_pack8(v, sc.inv);
        if ((threadIdx.x & 15) == 0) sl[r * nb + b] = sc.s;
      }
      __syncthreads();
      x[0] = reinterpret_cast<const uint8_t*>(rows_lds) + min(lr, rows - 1) * (K + 16) + lq * 16;
      xs[0] = sl + min(lr, rows - 1) * nb;
    }
    floatx4 acc[WF][RB];
#pragma unroll
    for (int f = 0; f < WF; ++f)
#pragma unroll
      for (int t = 0; t < RB; ++t) acc[f][t] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int kb = kw; kb < nkb; kb += ks) {
      if (kb != kw) load_weights(kb);
      v8i32 xv[RB];
      float sx[RB], sw[WF];
#pragma unroll
      for (int t = 0; t < RB; ++t) {
        xv[t] = load_codes(x[t], lq, kb * 128, K);
        sx[t] = xs[t][kb];
      }
#pragma unroll
      for (int f = 0; f < WF; ++f) sw[f] = ws[f][kb];
      Codes wc[WF];
#pragma unroll
      for (int f = 0; f < WF; ++f) wc[f] = widen(wv[f]);
#pragma unroll
      for (int t = 0; t < RB; ++t) {
        const Codes xc = widen(xv[t]);
#pragma unroll
        for (int f = 0; f < WF; ++f) {
          const floatx4 p = block_product(wc[f], xc);
          const float sc = sx[t] * sw[f];
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[f][t][q] = fmaf(p[q], sc, acc[f][t][q]);
        }
      }
    }
    if (ks > 1) {
      if (kw) {
#pragma unroll
        for (int f = 0; f < WF; ++f)
#pragma unroll
          for (int t = 0; t < RB; ++t)
            *reinterpret_cast<floatx4*>(&part[wave - wave / ks - 1][f][t][lane * 4]) = acc[f][t];
      }
      __syncthreads();
    }
    if (!kw && strip < strips) {
      const int p0 = wave - wave / ks;   // the first of the strip's ks - 1 parts
#pragma unroll
      for (int t = 0; t < RB; ++t) {
        for (int s = 0; s < ks - 1; ++s)
#pragma unroll
          for (int f = 0; f < WF; ++f)
            acc[f][t] += *reinterpret_cast<floatx4*>(&part[p0 + s][f][t][lane * 4]);
        const int r = 16 * t + lr;
        if (r >= rows) continue;
        const int nc = n0 + lq * 4;
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
    __syncthreads();   // LDS is free for the next item
  }
}

// Streams: the groups of a plan's thin experts (up to 16 rows at a time),
// quantised rows. A workgroup of eight waves walks eight strips of 16 weight
// rows (gate/up: 16 of each matrix, so a scale block of 128 features, which
// it quantises itself; down: 128 columns), ks waves sharing a strip's blocks
// of K, so that a workgroup's loads run through its weights in pieces of
// whole rows: a wave that walked its rows alone, 128 bytes of 16 rows at a
// time, got half of the rate. The rows' fragments stay in registers over all
// strips where K <= 128 ks NX. Bound by memory: 128 tokens on 129 experts, D
// 2048, F 768, take 83 us for gate/up (406 MB, 4.9 TB/s) and 49 for down (203
// MB, 4.1 TB/s; a workgroup lives for two steps, too few to hide its start).
// Loads without a place in the caches (nontemporal) were 7 % slower, the next
// step's loads a step earlier gained 2 us of down and lost 2 at K = 512.
template <int MODE, int NX>
__global__ __launch_bounds__(512, 4) void f8_stream_kernel(F8Args a, int ks) {
  constexpr int WF = MODE == 1 ? 2 : 1;
  __shared__ __attribute__((aligned(16))) float red[2][8][WF][256];
  __shared__ uint32_t mx[8][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int K = a.K, N = a.N, nkb = K / 128, nnb = N / 128;
  const uint32_t item = wide_block();
  const int gi = item / (uint32_t)nnb, cb = item - gi * (uint32_t)nnb;
  if (gi >= *a.groups) return;   // the whole workgroup, before any barrier
  const int32_t* g = a.list + 4 * (size_t)gi;
  const int e = g[0], rows = g[2], row0 = g[3];
  const int kw = wave & (ks - 1), ws = wave / ks, sw = 8 / ks;
  const int nch = (nkb + ks * NX - 1) / (ks * NX);   // chunks of K a strip
  const int steps = ks * nch;                        // ks batches of sw strips

  const size_t wbase = ((size_t)e * N + cb * 128 + lr) * K + lq * 16;
  const uint8_t* w0 = a.B0 + wbase;
  const uint8_t* w1 = MODE == 1 ? a.B1 + wbase : nullptr;
  v8i32 w[NX][WF];
  auto load_weights = [&](int st, int i) {
    const int it = nch == 1 ? st : st / nch, ch = st - it * nch;
    const int kb = min((ch * NX + i) * ks + kw, nkb - 1);
    const size_t off = (size_t)((it * sw + ws) * 16) * K + kb * 128;
    w[i][0] = load_codes(w0 + off);
    if (MODE == 1) w[i][WF - 1] = load_codes(w1 + off);
  };
  int64_t xr = row0 + min(lr, rows - 1);
#pragma unroll
  for (int i = 0; i < NX; ++i) load_weights(0, i);
  if (MODE == 1) xr = a.pair_token[xr];
  const uint8_t* x = a.A + (size_t)xr * K + lq * 16;
  const float* xs = a.As + (size_t)xr * nkb;
  const float* s0 = a.B0s + ((size_t)e * nnb + cb) * nkb;
  const float* s1 = MODE == 1 ? a.B1s + ((size_t)e * nnb + cb) * nkb : nullptr;
  v8i32 xv[NX];
  float sc[NX][WF];
  auto load_rows = [&](int ch) {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int kb = min((ch * NX + i) * ks + kw, nkb - 1);
      xv[i] = load_codes(x + kb * 128);
      const float sx = xs[kb];
      sc[i][0] = sx * s0[kb];
      if (MODE == 1) sc[i][WF - 1] = sx * s1[kb];
    }
  };
  floatx4 acc[WF];
  floatx4 mine[WF];   // the strip this wave finishes: strip `wave`
  for (int st = 0; st < steps; ++st) {
    const int it = nch == 1 ? st : st / nch, ch = st - it * nch;
    if (nch > 1 || st == 0) load_rows(ch);
    if (ch == 0) {
#pragma unroll
      for (int f = 0; f < WF; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const bool any = (ch * NX + i) * ks + kw < nkb;   // uniform in the wave
      if (any) {
        const Codes xc = widen(xv[i]);
#pragma unroll
        for (int f = 0; f < WF; ++f) {
          const floatx4 p = block_product(widen(w[i][f]), xc);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[f][q] = fmaf(p[q], sc[i][f], acc[f][q]);
        }
      }
      // the next step's weights into the registers just read: in flight over
      // the sums below
      if (st + 1 < steps) load_weights(st + 1, i);
    }
    if (ch < nch - 1) continue;
    // the ks partial sums of each strip meet in the wave of the strip's
    // number; a half of `red` is written again two barriers later
    float (*const half)[WF][256] = red[it & 1];
#pragma unroll
    for (int f = 0; f < WF; ++f) *reinterpret_cast<floatx4*>(&half[wave][f][lane * 4]) = acc[f];
    asm volatile("" ::: "memory");
    wait_vm_lgkm0<63>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (wave / sw == it) {
      const int p0 = (wave - it * sw) * ks;
#pragma unroll
      for (int f = 0; f < WF; ++f) {
        mine[f] = *reinterpret_cast<const floatx4*>(&half[p0][f][lane * 4]);
        for (int k = 1; k < ks; ++k)
          mine[f] += *reinterpret_cast<const floatx4*>(&half[p0 + k][f][lane * 4]);
      }
    }
  }
  const size_t row = (size_t)(row0 + lr);
  const int n0 = cb * 128 + wave * 16 + lq * 4;
  if constexpr (MODE == 1) {
    float h[4];
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      h[q] = swiglu(mine[0][q], mine[WF - 1][q], a.clamp);
      m = max(m, mag_bits(h[q]));
    }
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if (lq == 0) mx[wave][lr] = m;
    __syncthreads();
    m = mx[0][lr];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = max(m, mx[w][lr]);
    if (lr < rows) {
      const F8Scale fs = f8_scale(m);
      int o = 0;
      o = __builtin_amdgcn_cvt_pk_fp8_f32(h[0] * fs.inv, h[1] * fs.inv, o, false);
      o = __builtin_amdgcn_cvt_pk_fp8_f32(h[2] * fs.inv, h[3] * fs.inv, o, true);
      *reinterpret_cast<int*>(static_cast<uint8_t*>(a.out) + row * N + n0) = o;
      if (wave == 0 && lq == 0) a.out_s[row * nnb + cb] = fs.s;
    }
  } else if (lr < rows) {
    const float v[4] = {mine[0][0], mine[0][1], mine[0][2], mine[0][3]};
    store_out4(a.out, a.odt, row * N + n0, v);
  }
}

template <int MODE, int NX>
static void run_stream(const F8Args& a, int ks, int64_t grid, hipStream_t s) {
  hipLaunchKernelGGL((f8_stream_kernel<MODE, NX>), wide_grid(grid), dim3(512), 0, s, a, ks);
}

hipError_t launch_f8_stream(const F8Args& a, hipStream_t s) {
  const int64_t grid = (int64_t)a.max_groups * (a.N / 128);
  if (grid == 0) return hipSuccess;
  // The most waves a strip that leave each two blocks or more (one or more: 56
  // us, not 52, for the down stream of 128 tokens, K = 768), two or three
  // blocks a wave and chunk, whichever leaves fewer idle (two at K = 768: 74
  // us, not 52; six, and one wave a strip: 92).
  const int nkb = a.K / 128;
  int ks = 8;
  while (ks > 1 && nkb < 2 * ks) ks >>= 1;
  const bool three = (nkb + ks * 2 - 1) / (ks * 2) * 2 > (nkb + ks * 3 - 1) / (ks * 3) * 3 - 1;
  if (a.mode == 1) run_stream<1, 2>(a, ks, grid, s);
  else if (three) run_stream<2, 3>(a, ks, grid, s);
  else run_stream<2, 2>(a, ks, grid, s);
  return hipGetLastError();
}

static size_t strip_lds(int rows, int K) { return (size_t)rows * (K + 16 + K / 128 * 4); }

bool f8_strip_raw_fits(int rows, int K) { return rows <= 16 && strip_lds(rows, K) <= kStripLds; }

template <int MODE, int RB, int SRC>
static void run_strip(const F8Args& a, unsigned grid, hipStream_t s) {
  const size_t lds = SRC ? strip_lds(a.lds_rows, a.K) : 0;
  hipLaunchKernelGGL((f8_strip_kernel<MODE, RB, SRC>), dim3(grid), dim3(256), lds, s, a);
}

hipError_t launch_f8_strip(const F8Args& a, int ncu, hipStream_t s) {
  const int spw = 4 / strip_share((a.K + 127) / 128);
  const int64_t sblocks = (((int64_t)a.N + 15) / 16 + spw - 1) / spw;
  // 64 rows a workgroup once 16 would make four workgroups a CU: weights are
  // read a fourth as often, by fewer waves (us with 64 / 16 rows: 64 rows by
  // 4096 x 4096 17.6 / 22.0, by 2048 x 1024 7.5 / 5.8; 128 by 1001 x 1040 7.7
  // / 5.7; 517 by 1001 x 1040 10.4 / 10.7)
  const int64_t groups16 = a.mode == 0 ? (a.M + 15) / 16 : a.max_groups;
  const int rb = a.mode == 0 && a.M > 16 && groups16 * sblocks >= 4 * ncu ? 4 : 1;
  const int64_t items = (groups16 + rb - 1) / rb * sblocks;
  if (items == 0) return hipSuccess;
  const unsigned grid = (unsigned)std::min<int64_t>(items, (int64_t)ncu * 16);
  if (a.mode == 0 && rb == 1) run_strip<0, 1, 0>(a, grid, s);
  else if (a.mode == 0) run_strip<0, 4, 0>(a, grid, s);
  else if (a.mode == 1) run_strip<1, 1, 1>(a, grid, s);
  else run_strip<2, 1, 1>(a, grid, s);
  return hipGetLastError();
}

}  // namespace moe
