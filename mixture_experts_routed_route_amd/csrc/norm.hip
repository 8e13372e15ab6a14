// RMS norms after a block and before the next one, fused with the block's
// gate and the residual's scale, on gfx950.
//
//   z  = u / rms(u) * p        (post-norm; without one z = u)
//   r' = r + alpha * g * z     (g one value a channel or a token, or none)
//   x  = r' / rms(r') * w      (pre-norm of the next block, from the f32 r')
//   rms(v) = sqrt(mean(v^2) + eps)
//
// Every value is read once and written once: a row lives in the registers
// of the threads that own it between the two sums, so the launch is bound
// by HBM. A row takes 64 threads (four rows a workgroup) or a workgroup of
// up to 1024, 8 or 16 values each, so that a thread's registers leave
// several workgroups a CU, whose loads cover one another's sums.
#include <algorithm>

#include "rows_common.h"

namespace moe {

namespace {

// threads of one row's sums, and rows of one workgroup
template <int TPR> struct RowShape {
  static constexpr int kRows = TPR == 64 ? 4 : 1;
  static constexpr int kThreads = TPR * kRows;
};

__device__ __forceinline__ float param(float v, int unit) { return unit ? 1.f + v : v; }

}  // namespace

template <int TPR, int NV>
__global__ __launch_bounds__(RowShape<TPR>::kThreads) void norm_forward_kernel(NormArgs a) {
  __shared__ float sh[2 * 16];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RowShape<TPR>::kRows + threadIdx.x / TPR;
  if (row >= a.T) return;   // whole waves, and whole workgroups where TPR > 64
  const size_t base = (size_t)row * a.D;
  Raw8 rr[NV], ur[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * 8;
    if (c < a.D) {
      rr[i] = load_raw8(a.r, a.rdt, base + c);
      if (a.u) ur[i] = load_raw8(a.u, a.udt, base + c);
    }
  }
  float r[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * TPR + t) * 8 < a.D) {
      raw8_to_f32(rr[i], a.rdt, r[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] = 0.f;
    }
  }
  if (a.u) {
    float u[NV][8], ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * TPR + t) * 8 < a.D) {
        raw8_to_f32(ur[i], a.udt, u[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] = 0.f;
      }
    }
    float inv = 1.f;
    if (a.p) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] = fmaf(u[i][j], u[i][j], ss[0]);
      row_sums<TPR>(ss, sh);
      inv = rsqrtf(ss[0] / (float)a.D + a.eps);
    }
    float gt = a.alpha;
    if (a.g && a.gate_token) {
      float one;
      if (a.gdt == MOE_F32) one = static_cast<const float*>(a.g)[row];
      else if (a.gdt == MOE_BF16) one = (float)static_cast<const __bf16*>(a.g)[row];
      else one = (float)static_cast<const _Float16*>(a.g)[row];
      gt *= one;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * 8;
      if (c < a.D) {
        float pv[8], gv[8];
        if (a.p) raw8_to_f32(load_raw8(a.p, a.wdt, c), a.wdt, pv);
        if (a.g && !a.gate_token) raw8_to_f32(load_raw8(a.g, a.gdt, c), a.gdt, gv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float z = u[i][j];
          if (a.p) z = z * inv * param(pv[j], a.unit);
          if (a.g && !a.gate_token) z *= gv[j];
          r[i][j] = fmaf(gt, z, r[i][j]);
        }
        store8(a.r_out, a.rdt, base + c, r[i]);
      }
    }
  }
  if (!a.w) return;
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss[0] = fmaf(r[i][j], r[i][j], ss[0]);
  row_sums<TPR>(ss, sh + 16);
  const float inv = rsqrtf(ss[0] / (float)a.D + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * 8;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < a.D) {
      float wv[8];
      raw8_to_f32(load_raw8(a.w, a.wdt, c), a.wdt, wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = r[i][j] * inv * param(wv[j], a.unit);
      if (a.xdt != MOE_F8B128) store8(a.x, a.xdt, base + c, x);
    }
    if (a.xdt == MOE_F8B128) {
      // 16 neighbouring lanes hold one block of the row
      const F8Scale sc = f8_scale(max16(mag_max8(x)));
      if (c < a.D) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.x) + base + c) = f8_pack8(x, sc.inv);
        if ((t & 15) == 0) a.xs[(size_t)row * a.nb + (c >> 7)] = sc.s;
      }
    }
  }
}

template <int TPR, int NV>
static hipError_t run_norm_forward(const NormArgs& a, hipStream_t s) {
  constexpr int R = RowShape<TPR>::kRows;
  hipLaunchKernelGGL((norm_forward_kernel<TPR, NV>), dim3((unsigned)(((int64_t)a.T + R - 1) / R)),
                     dim3(RowShape<TPR>::kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  if (a.D <= 512) return run_norm_forward<64, 1>(a, s);
  if (a.D <= 1024) return run_norm_forward<64, 2>(a, s);
  if (a.D <= 2048) return run_norm_forward<256, 1>(a, s);
  if (a.D <= 4096) return run_norm_forward<256, 2>(a, s);
  if (a.D <= 8192) return run_norm_forward<512, 2>(a, s);
  return run_norm_forward<1024, 2>(a, s);
}

// ---- backward ---------------------------------------------------------------
//
// With n = r' inv, t = dx w, m = mean(t n):      (sums over a row's D values)
//   d   = dr' + inv (t - n m)        the gradient of r', and of r
//   dw += dx n
//   dz  = alpha g d,  dg += alpha d z
// and with v = u inv_u, tp = dz p, mp = mean(tp v):
//   du  = inv_u (tp - v mp),  dp += dz v      (without a post-norm du = dz)
// The inverse norms are recomputed from r' and u, which are read anyway. A
// workgroup walks rows gridDim.x apart and holds its partial sums of dw, dp
// and a channel gate's dg in registers; it writes them once, [3][grid][D],
// and a second launch adds the workgroups' partials in order (no atomics:
// the same bits from run to run).
template <int TPR, int NV>
__global__ __launch_bounds__(RowShape<TPR>::kThreads) void norm_backward_kernel(NormBwdArgs a) {
  __shared__ float sh[2][5 * 16];
  const int t = threadIdx.x % TPR;
  const int sub = threadIdx.x / TPR;
  constexpr int R = RowShape<TPR>::kRows;
  const float invD = 1.f / (float)a.D;
  float dw[NV][8], dp[NV][8], dg[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = dp[i][j] = dg[i][j] = 0.f;
  const bool gate_ch = a.g && !a.gate_token;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * R + sub; row < a.T; row += (int64_t)gridDim.x * R) {
    // Between two rows' uses of one half of sh lies a barrier that every wave
    // reaches after its reads: the second sum's where there is a block, else
    // the next row's (the halves then take turns).
    float* const sh0 = sh[a.u ? 0 : turn];
    turn ^= 1;
    const size_t base = (size_t)row * a.D;
    Raw8 r8[NV], x8[NV], u8[NV], e8[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * 8;
      if (c < a.D) {
        if (a.w) {
          r8[i] = load_raw8(a.r, a.rdt, base + c);
          x8[i] = load_raw8(a.dx, a.dxdt, base + c);
        }
        if (a.u) u8[i] = load_raw8(a.u, a.udt, base + c);
        if (a.dr) e8[i] = load_raw8(a.dr, a.rdt, base + c);
      }
    }
    float sum[3] = {0.f, 0.f, 0.f};   // r'^2, t r', u^2
    float r[NV][8], dx[NV][8], u[NV][8], d[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] = dx[i][j] = u[i][j] = d[i][j] = 0.f;
      if (c < a.D) {
        if (a.w) {
          raw8_to_f32(r8[i], a.rdt, r[i]);
          raw8_to_f32(x8[i], a.dxdt, dx[i]);
          float wv[8];
          raw8_to_f32(load_raw8(a.w, a.wdt, c), a.wdt, wv);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sum[0] = fmaf(r[i][j], r[i][j], sum[0]);
            sum[1] = fmaf(dx[i][j] * param(wv[j], a.unit), r[i][j], sum[1]);
          }
        }
        if (a.u) raw8_to_f32(u8[i], a.udt, u[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[2] = fmaf(u[i][j], u[i][j], sum[2]);
        if (a.dr) raw8_to_f32(e8[i], a.rdt, d[i]);
      }
    }
    row_sums<TPR>(sum, sh0);
    const float inv = rsqrtf(sum[0] * invD + a.eps);
    const float m = sum[1] * inv * inv * invD;   // mean(t n) inv
    const float inv_u = a.p ? rsqrtf(sum[2] * invD + a.eps) : 1.f;
    float gt = a.alpha;
    if (a.g && a.gate_token) {
      if (a.gdt == MOE_F32) gt *= static_cast<const float*>(a.g)[row];
      else if (a.gdt == MOE_BF16) gt *= (float)static_cast<const __bf16*>(a.g)[row];
      else gt *= (float)static_cast<const _Float16*>(a.g)[row];
    }
    float s2[2] = {0.f, 0.f};   // tp u, d z
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * 8;
      if (c < a.D) {
        if (a.w) {
          float wv[8];
          raw8_to_f32(load_raw8(a.w, a.wdt, c), a.wdt, wv);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            dw[i][j] = fmaf(dx[i][j], r[i][j] * inv, dw[i][j]);
            d[i][j] += inv * (dx[i][j] * param(wv[j], a.unit) - r[i][j] * m);
          }
        }
        store8(a.dr_out, a.rdt, base + c, d[i]);
        if (a.u) {
          float pv[8], gv[8];
          if (a.p) raw8_to_f32(load_raw8(a.p, a.wdt, c), a.wdt, pv);
          if (gate_ch) raw8_to_f32(load_raw8(a.g, a.gdt, c), a.gdt, gv);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float v = u[i][j] * inv_u;
            const float pj = a.p ? param(pv[j], a.unit) : 1.f;
            if (gate_ch) dg[i][j] = fmaf(a.alpha * d[i][j], v * pj, dg[i][j]);
            if (a.gate_token) s2[1] = fmaf(d[i][j], v * pj, s2[1]);
            const float dz = gt * d[i][j] * (gate_ch ? gv[j] : 1.f);
            dp[i][j] = fmaf(dz, v, dp[i][j]);
            d[i][j] = dz * pj;
            s2[0] = fmaf(d[i][j], v, s2[0]);
          }
        }
      }
    }
    if (a.u) {
      row_sums<TPR>(s2, sh[1]);
      const float mp = a.p ? s2[0] * invD : 0.f;
      if (a.dg_token && t == 0) a.dg_token[row] = a.alpha * s2[1];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * 8;
        if (c < a.D) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            o[j] = a.p ? inv_u * (d[i][j] - u[i][j] * inv_u * mp) : d[i][j];
          store8(a.du, a.udt, base + c, o);
        }
      }
    }
  }
  // this row slot's partials: slot blockIdx.x * R + sub of grid * R
  const size_t slots = (size_t)gridDim.x * R;
  const size_t slot = (size_t)blockIdx.x * R + sub;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * 8;
    if (c < a.D) {
      if (a.w) store8(a.part, MOE_F32, slot * a.D + c, dw[i]);
      if (a.p) store8(a.part, MOE_F32, (slots + slot) * a.D + c, dp[i]);
      if (gate_ch) store8(a.part, MOE_F32, (2 * slots + slot) * a.D + c, dg[i]);
    }
  }
}

// out[c] = the slots' partials of column c, added in a fixed order: 16
// threads take every 16th slot, then their sums in order. blockIdx.y picks
// the vector.
__global__ __launch_bounds__(256) void norm_columns_kernel(
    const float* __restrict__ part, int slots, int D, float* o0, float* o1, float* o2) {
  __shared__ float sh[16][17];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int c = blockIdx.x * 16 + (threadIdx.x & 15);
  const int g = threadIdx.x >> 4;
  float s = 0.f;
  if (c < D)
    for (int k = g; k < slots; k += 16) s += part[((size_t)blockIdx.y * slots + k) * D + c];
  sh[g][threadIdx.x & 15] = s;
  __syncthreads();
  if (g == 0 && c < D) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) v += sh[k][threadIdx.x & 15];
    out[c] = v;
  }
}

namespace {

struct BwdShape { int grid, slots; };
constexpr int kBwdGrid = 512;   // two workgroups a compute unit
BwdShape bwd_shape(int T, int D) {
  const int rows = D <= 1024 ? 4 : 1;
  const int64_t need = ((int64_t)T + rows - 1) / rows;
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(need, kBwdGrid));
  return {grid, grid * rows};
}

}  // namespace

size_t norm_backward_part_floats(int T, int D) {
  return (size_t)3 * bwd_shape(T, D).slots * D;
}

template <int TPR, int NV>
static void run_norm_backward(const NormBwdArgs& a, int grid, hipStream_t s) {
  hipLaunchKernelGGL((norm_backward_kernel<TPR, NV>), dim3(grid),
                     dim3(RowShape<TPR>::kThreads), 0, s, a);
}

hipError_t launch_norm_backward(const NormBwdArgs& a, hipStream_t s) {
  const BwdShape sh = bwd_shape(a.T, a.D);
  if (a.D <= 512) run_norm_backward<64, 1>(a, sh.grid, s);
  else if (a.D <= 1024) run_norm_backward<64, 2>(a, sh.grid, s);
  else if (a.D <= 2048) run_norm_backward<256, 1>(a, sh.grid, s);
  else if (a.D <= 4096) run_norm_backward<256, 2>(a, sh.grid, s);
  else if (a.D <= 8192) run_norm_backward<512, 2>(a, sh.grid, s);
  else run_norm_backward<1024, 2>(a, sh.grid, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_columns_kernel, dim3((a.D + 15) / 16, 3), dim3(256), 0, s, a.part,
                     sh.slots, a.D, a.dw, a.p ? a.dp : nullptr, a.dg_channel);
  return hipGetLastError();
}

}  // namespace moe
