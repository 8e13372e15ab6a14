// Quantisers of the 8-bit block format (MOE_F8B128) on gfx950: rows with a
// scale per row and 128 values, weights with a scale per 128 x 128 block.
// The arithmetic is in rows_common.h (f8_scale, f8_pack8).
#include "rows_common.h"

namespace moe {

// Rows. 16 neighbouring lanes own one block of 128 values, 8 each: one pass
// over the data, the block's largest magnitude from four exchanges.
__global__ __launch_bounds__(256) void quant_rows_kernel(
    const void* __restrict__ x, int dt, uint32_t n_blocks, uint32_t nb, int K,
    uint8_t* __restrict__ q, float* __restrict__ s) {
  const uint32_t g = wide_block() * 16u + (threadIdx.x >> 4);
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

hipError_t launch_quant_rows(const void* x, int dt, int64_t rows, int K,
                             void* q, float* s, hipStream_t st) {
  const int64_t nb = (K + 127) / 128;
  const int64_t n = rows * nb;
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(quant_rows_kernel, wide_grid((n + 15) / 16), dim3(256), 0, st,
                     x, dt, (uint32_t)n, (uint32_t)nb, K, (uint8_t*)q, s);
  return hipGetLastError();
}

// Weights: a workgroup takes one 128 x 128 block, 16 rows a pass with 16
// lanes a row, all of it in registers between the maximum and the codes.
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
  const int64_t nn = (N + 127) / 128, nk = (K + 127) / 128;
  const int64_t n = mats * nn * nk;
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(quant_weights_kernel, wide_grid(n), dim3(256), 0, st, w, dt,
                     (uint32_t)n, (uint32_t)nn, (uint32_t)nk, N, K, (uint8_t*)q, s);
  return hipGetLastError();
}

}  // namespace moe
