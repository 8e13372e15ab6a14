// Quantisers of the 8-bit block format (MOE_F8B128) on gfx950: rows with a
// scale per row and 128 values, weights with a scale per 128 x 128 block.
// The arithmetic is in rows_common.h (f8_scale, f8_pack8).
#include "rows_common.h"

namespace moe {

// Rows. 16 neighbouring lanes own one block of 128 values, 8 each: one pass
// over the data, the block's largest magnitude from four exchanges. Bound by
// memory: 13312 x 4096 f16 in 31 us, 5.4 TB/s.
__device__ __forceinline__ void quant_blocks(
    uint32_t workgroup, const void* __restrict__ x, int dt, uint32_t n_blocks, uint32_t nb, int K,
    uint8_t* __restrict__ q, float* __restrict__ s) {
  const uint32_t g = workgroup * 16u + (threadIdx.x >> 4);
  if (g >= n_blocks) return;   // whole groups of 16 lanes
  const uint32_t row = g / nb, b = g - row * nb;
  const int k = (int)(b * 128u) + (threadIdx.x & 15) * 8;
  const size_t at = (size_t)row * K + k;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (k < K) raw8_to_f32(load_raw8(x, dt, at), dt, v);
  const F8Scale sc = f8_scale(max16(mag_max8(v)));
  if (k < K) *reinterpret_cast<uint2*>(q + at) = f8_pack8(v, sc.inv);
  if ((threadIdx.x & 15) == 0) s[g] = sc.s;
}

__global__ __launch_bounds__(256) void quant_rows_kernel(
    const void* __restrict__ x, int dt, uint32_t n_blocks, uint32_t nb, int K,
    uint8_t* __restrict__ q, float* __restrict__ s) {
  quant_blocks(wide_block(), x, dt, n_blocks, nb, K, q, s);
}

hipError_t launch_quant_rows(const void* x, int dt, int64_t rows, int K,
                             void* q, float* s, hipStream_t st) {
  const int64_t nb = ((int64_t)K + 127) / 128;
  const int64_t n = rows * nb;
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(quant_rows_kernel, wide_grid((n + 15) / 16), dim3(256), 0, st,
                     x, dt, (uint32_t)n, (uint32_t)nb, K, (uint8_t*)q, s);
  return hipGetLastError();
}

// A layer's first launch: x's rows quantised, and beside them, in the first
// workgroup, the plan's work lists. Experts of at most thin_rows rows are cut
// into parts of 16 rows, in expert order; the others into tiles of 256, the
// experts of most rows first (ties: the lower index). As two launches they
// took 5 us more; 4096 tokens x 2048 on 128 experts take 9 us.
__global__ __launch_bounds__(256) void f8_prepare_kernel(F8PrepareArgs a, uint32_t n_blocks) {
  constexpr int kPad = (kMaxExperts + 1 + 3) / 4 * 4;
  __shared__ __attribute__((aligned(16))) int tall[kPad];   // rows of a tile expert, else -1
  __shared__ int order[kPad];
  __shared__ int sums[2][4];
  if (blockIdx.x) {
    quant_blocks(blockIdx.x - 1, a.x, a.xdt, n_blocks, (uint32_t)a.D / 128, a.D, a.q, a.s);
    return;
  }
  // thread t's exclusive sum of v over the threads, and the total; the two
  // halves of `sums` take turns
  int turn = 0;
  auto scan = [&](int v, int* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 63) sums[turn][wave] = incl;
    __syncthreads();
    int pre = 0, tot = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < wave) pre += sums[turn][i];
      tot += sums[turn][i];
    }
    turn ^= 1;
    *total = tot;
    return pre + incl - v;
  };
  const int n = a.n_exp, n4 = (n + 3) / 4 * 4;
  int parts = 0, n_tall = 0;
  for (int b = 0; b < n; b += 256) {
    const int e = b + (int)threadIdx.x;
    const int c = e < n ? a.counts[e] : 0;
    const int first = e < n ? a.offsets[e] : 0;
    const bool thin = c <= a.thin_rows;
    if (e < n4) tall[e] = thin ? -1 : c;
    const int mine = thin ? (c + 15) / 16 : 0;
    int all;
    const int at = parts + scan(mine, &all);
    for (int i = 0; i < mine; ++i) {
      int32_t* p = a.parts + 4 * (size_t)(at + i);
      p[0] = e;
      p[1] = 16 * i;
      p[2] = min(16, c - 16 * i);
      p[3] = first + 16 * i;
    }
    parts += all;
    scan(thin ? 0 : 1, &all);
    n_tall += all;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n && n_tall; e += 256) {
    const int c = tall[e];
    if (c < 0) continue;
    int rank = 0;
    for (int f = 0; f < n4; f += 4) {
      const int4 v = *reinterpret_cast<const int4*>(&tall[f]);
      rank += (v.x > c || (v.x == c && f + 0 < e)) + (v.y > c || (v.y == c && f + 1 < e)) +
              (v.z > c || (v.z == c && f + 2 < e)) + (v.w > c || (v.w == c && f + 3 < e));
    }
    order[rank] = e;
  }
  __syncthreads();
  int tiles = 0;
  for (int b = 0; b < n_tall; b += 256) {
    const int r = b + (int)threadIdx.x;
    const int e = r < n_tall ? order[r] : 0;
    const int mine = r < n_tall ? (tall[e] + kFullBM - 1) / kFullBM : 0;
    int all;
    const int at = tiles + scan(mine, &all);
    for (int i = 0; i < mine; ++i) {
      a.tiles[2 * (size_t)(at + i)] = e;
      a.tiles[2 * (size_t)(at + i) + 1] = i * kFullBM;
    }
    tiles += all;
  }
  if (threadIdx.x == 0) {
    a.meta[kF8Parts] = parts;
    a.meta[kF8Tiles] = tiles;
  }
}

hipError_t launch_f8_prepare(const F8PrepareArgs& a, hipStream_t st) {
  // T D stays below 2^31: fewer than 2^20 workgroups
  const uint32_t n = (uint32_t)((int64_t)a.T * (a.D / 128));
  hipLaunchKernelGGL(f8_prepare_kernel, dim3((n + 15) / 16 + 1), dim3(256), 0, st, a, n);
  return hipGetLastError();
}

// Weights: a workgroup takes one 128 x 128 block, 16 rows a pass with 16
// lanes a row, all of it in registers between the maximum and the codes. Bound
// by memory: 128 x 768 x 2048 bf16 in 130 us, 4.7 TB/s; one matrix of 4096 x
// 4096 in 11.
__global__ __launch_bounds__(256) void quant_weights_kernel(
    const void* __restrict__ w, int dt, uint32_t n_blocks, uint32_t nn, uint32_t nk, int N,
    int K, uint8_t* __restrict__ q, float* __restrict__ s) {
  __shared__ uint32_t mx[4];
  const uint32_t blk = wide_block();
  if (blk >= n_blocks) return;   // whole workgroups
  const uint32_t kb = blk % nk, t = blk / nk;
  const uint32_t rb = t % nn, mat = t / nn;
  const int k = (int)kb * 128 + (threadIdx.x & 15) * 8;
  const int r0 = (int)rb * 128 + (threadIdx.x >> 4);
  const size_t base = (size_t)mat * N * K;
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (k < K && r < N) {
      raw8_to_f32(load_raw8(w, dt, base + (size_t)r * K + k), dt, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
    m = max(m, mag_max8(v[i]));
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
  if ((threadIdx.x & 63) == 0) mx[threadIdx.x >> 6] = m;
  __syncthreads();
  const F8Scale sc = f8_scale(max(max(mx[0], mx[1]), max(mx[2], mx[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (k < K && r < N)
      *reinterpret_cast<uint2*>(q + base + (size_t)r * K + k) = f8_pack8(v[i], sc.inv);
  }
  if (threadIdx.x == 0) s[blk] = sc.s;
}

hipError_t launch_quant_weights(const void* w, int dt, int64_t mats, int N,
                                int K, void* q, float* s, hipStream_t st) {
  const int64_t nn = ((int64_t)N + 127) / 128, nk = ((int64_t)K + 127) / 128;
  const int64_t n = mats * nn * nk;
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(quant_weights_kernel, wide_grid(n), dim3(256), 0, st, w, dt,
                     (uint32_t)n, (uint32_t)nn, (uint32_t)nk, N, K, (uint8_t*)q, s);
  return hipGetLastError();
}

}  // namespace moe
