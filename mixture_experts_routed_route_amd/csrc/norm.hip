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
// several workgroups a CU, whose loads cover one another's sums. Forward: 13312
// x 4096, f32 residual, f16 block and x, 120 us, 5.4 TB/s (a copy of 1 GiB runs
// at 5.1, an addition in place at 5.9).
#include <algorithm>

#include "rows_common.h"

namespace moe {

namespace {

// threads of one row's sums, and rows of one workgroup
template <int TPR> struct RowShape {
  static constexpr int kRows = TPR == 64 ? 4 : 1;
  static constexpr int kThreads = TPR * kRows;
};

__device__ __forceinline__ float load_one(const void* p, int dt, size_t i) {
  if (dt == MOE_F32) return static_cast<const float*>(p)[i];
  if (dt == MOE_BF16) return (float)static_cast<const __bf16*>(p)[i];
  return (float)static_cast<const _Float16*>(p)[i];
}

__device__ __forceinline__ float param(float v, int unit) { return unit ? 1.f + v : v; }

}  // namespace

template <int TPR, int NV>
__global__ __launch_bounds__(RowShape<TPR>::kThreads) void norm_forward_kernel(NormArgs a) {
  __shared__ float sh[2 * 16];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)wide_block() * RowShape<TPR>::kRows + threadIdx.x / TPR;
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
      gt *= load_one(a.g, a.gdt, row);
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
  hipLaunchKernelGGL((norm_forward_kernel<TPR, NV>), wide_grid(((int64_t)a.T + R - 1) / R),
                     dim3(RowShape<TPR>::kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  // 8 values a thread where they fill 256 or 512 threads, 16 a thread else.
  // 13312 x 4096 f32 residual and f16 block, us of the same bytes as rows of
  // 1024 / 2048 / 4096 / 8192 values: this rule 126 / 122 / 123 / 131, twice
  // the values a thread (half at 1024 and 8192) 122 / 129 / 130 / 129, four
  // times - / 137 / 142 / 141.
  if (a.D <= 512) return run_norm_forward<64, 1>(a, s);
  if (a.D <= 1024) return run_norm_forward<64, 2>(a, s);
  if (a.D <= 2048) return run_norm_forward<256, 1>(a, s);
  if (a.D <= 4096) return run_norm_forward<512, 1>(a, s);
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
// d is linear in dr', t and r', so with a = alpha g p the second norm's sum
// of a u d is s3 + inv (s4 - inv^2 s1 / D s5) of the sums of a u dr', a u t
// and a u r': all six sums of a row are known after one pass and one barrier,
// and everything behind it is elementwise. The inverse norms are recomputed
// from r' and u, which are read anyway. A workgroup walks rows (R at a time),
// the parameters in LDS, the next row's loads in flight, its partial sums of
// dw, dp and a channel gate's dg in registers; it writes them once,
// [3][grid][D], and a second launch adds the workgroups' partials in order
// (no atomics: the same bits from run to run). 4096 x 2048 f32: 41 us and 4
// for the columns, 201 MB at 4.4 TB/s; 8192 x 8192 bf16 170 us, 4.7 TB/s: the
// walk's one barrier a row and the first and last rows' latency are left.
// Every load and store of the walk is a buffer instruction that is always
// there: what a type, a missing tensor, a short row or a row past the last
// leaves out lies past its buffer's end (loads give 0, stores write nothing).
// One counter orders loads and stores, and with branches between them the
// wait for a row's loads would cover the stores of the row before.
// SPLIT: rows of more than 8192 values, whose sums a launch of their own has
// left in `stats`; blockIdx.y walks a part of the columns (held whole, such a
// row's partial sums and values spilled: 4096 x 16384 bf16 in 1037 us, not
// 308).
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
constexpr int kPastEnd = (int)0x80000000u;

// eight values, f32 or 16-bit, as loaded
struct Wide8 { u32x4 a, b; };

__device__ __forceinline__ void wide_to_f32(const Wide8& w, int dt, float (&v)[8]) {
  if (dt == MOE_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(w.a[i]);
      v[4 + i] = __uint_as_float(w.b[i]);
    }
  } else if (dt == MOE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w.a[i] << 16);
      v[2 * i + 1] = __uint_as_float(w.a[i] & 0xFFFF0000u);
    }
  } else {
    const half8 h = __builtin_bit_cast(half8, w.a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  }
}

__device__ __forceinline__ Wide8 wide_from_f32(const float (&v)[8], int dt) {
  Wide8 w;
  if (dt == MOE_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w.a[i] = __float_as_uint(v[i]);
      w.b[i] = __float_as_uint(v[4 + i]);
    }
  } else if (dt == MOE_BF16) {
    bf16x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
    w.a = w.b = __builtin_bit_cast(u32x4, o);
  } else {
    half8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (_Float16)v[i];
    w.a = w.b = __builtin_bit_cast(u32x4, o);
  }
  return w;
}

// what a row's six sums (norm_backward_kernel) give: its inverse norms, mean(t
// n) inv, the second norm's mean, a token gate's gradient
struct RowStats { float inv, m, inv_u, mp, dg; };
__device__ __forceinline__ RowStats row_stats(const NormBwdArgs& a, const float (&sum)[6],
                                              float gt) {
  const float invD = 1.f / (float)a.D;
  RowStats s;
  s.inv = rsqrtf(sum[0] * invD + a.eps);
  s.m = sum[1] * s.inv * s.inv * invD;
  s.inv_u = a.p ? rsqrtf(sum[2] * invD + a.eps) : 1.f;
  const float aud = a.w ? sum[3] + s.inv * (sum[4] - s.m * sum[5]) : sum[3];
  s.mp = gt * s.inv_u * aud * invD;
  s.dg = s.inv_u * aud;
  return s;
}

// eight of the parameters k (0 w, 1 p, 2 alpha times a channel gate) from
// channel c; ones where there is none, zeros past the row
__device__ __forceinline__ void read_params(const NormBwdArgs& a, int k, int c, float (&v)[8]) {
  const void* src = k == 0 ? a.w : k == 1 ? a.p : a.gate_token ? nullptr : a.g;
  const int dt = k == 2 ? a.gdt : a.wdt;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = c < a.D ? 1.f : 0.f;
  if (src && c < a.D) {
    raw8_to_f32(load_raw8(src, dt, c), dt, v);
    if (k != 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = param(v[j], a.unit);
    }
  }
  if (k == 2) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= a.alpha;
  }
}

// the sums of rows of more than 8192 values, a workgroup a row:
// (inv, m, inv_u, mp) and a token gate's gradient
__global__ __launch_bounds__(1024) void norm_sums_kernel(NormBwdArgs a, float4* stats) {
  __shared__ float sh[6 * 16];
  const int64_t row = wide_block();
  if (row >= a.T) return;   // whole workgroups
  const size_t base = (size_t)row * a.D;
  float sum[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int c = threadIdx.x * 8; c < a.D; c += 8192) {
    float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float dx[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.w) {
      raw8_to_f32(load_raw8(a.r, a.rdt, base + c), a.rdt, r);
      raw8_to_f32(load_raw8(a.dx, a.dxdt, base + c), a.dxdt, dx);
    }
    if (a.u) raw8_to_f32(load_raw8(a.u, a.udt, base + c), a.udt, u);
    if (a.dr) raw8_to_f32(load_raw8(a.dr, a.rdt, base + c), a.rdt, d);
    float wv[8], pv[8], gv[8];
    read_params(a, 0, c, wv);
    read_params(a, 1, c, pv);
    read_params(a, 2, c, gv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float tt = dx[j] * wv[j], au = gv[j] * pv[j] * u[j];
      sum[0] = fmaf(r[j], r[j], sum[0]);
      sum[1] = fmaf(tt, r[j], sum[1]);
      sum[2] = fmaf(u[j], u[j], sum[2]);
      sum[3] = fmaf(au, d[j], sum[3]);
      sum[4] = fmaf(au, tt, sum[4]);
      sum[5] = fmaf(au, r[j], sum[5]);
    }
  }
  row_sums<1024>(sum, sh);
  if (threadIdx.x) return;
  const RowStats s = row_stats(a, sum, a.g && a.gate_token ? load_one(a.g, a.gdt, row) : 1.f);
  stats[row] = float4{s.inv, s.m, s.inv_u, s.mp};
  if (a.dg_token) a.dg_token[row] = s.dg;
}

template <int TPR, int R, int NV, bool SPLIT>
__global__ __launch_bounds__(TPR * R, NV == 1 ? 4 : 2) void norm_backward_kernel(
    NormBwdArgs a, const float4* stats) {
  constexpr int W = TPR / 64;   // waves a row
  extern __shared__ __attribute__((aligned(16))) float par[];   // [3][cols]: w, p, alpha p g
  __shared__ float sh[2][R][6 * W];
  __shared__ float fold[R > 1 ? (R - 1) * TPR * 8 : 1];
  constexpr int cols = TPR * NV * 8;
  const int t = threadIdx.x % TPR;
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);   // whole waves
  const int c0 = SPLIT ? (int)blockIdx.y * cols : 0;   // the first channel
  const bool gate_ch = a.g && !a.gate_token;
  const uint32_t u_values = a.u ? (uint32_t)a.D : 0u, w_values = a.w ? (uint32_t)a.D : 0u;
  // parameters h .. h + 3 of a thread's eight: four at a time, the loops over
  // halves kept apart, so that no more of them take registers
  auto params = [&](int k, int c, int h, float (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = par[k * cols + c + h + j];
  };
  for (int c = threadIdx.x * 8; c < cols; c += TPR * R * 8) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      float v[8];
      read_params(a, k, c0 + c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) par[k * cols + c + j] = v[j];
    }
  }
  float dw[NV][8], dp[NV][8], dg[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = dp[i][j] = dg[i][j] = 0.f;
  // a row of a tensor of `values` values a row (0: none)
  auto row_of = [&](const void* p, int dt, int64_t row, uint32_t values) {
    const int sz = dt == MOE_F32 ? 4 : 2;
    const bool live = row < a.T;
    return make_rsrc(static_cast<const char*>(p) + (size_t)(live ? row : 0) * a.D * sz,
                     live ? values * sz : 0u);
  };
  auto load8 = [&](__amdgpu_buffer_rsrc_t rs, int dt, int i) {
    const int off = (c0 + (i * TPR + t) * 8) * (dt == MOE_F32 ? 4 : 2);
    Wide8 w;
    w.a = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
    w.b = __builtin_amdgcn_raw_buffer_load_b128(rs, dt == MOE_F32 ? off + 16 : kPastEnd, 0, 0);
    return w;
  };
  auto put8 = [&](__amdgpu_buffer_rsrc_t rs, int dt, int i, const float (&v)[8]) {
    const int off = (c0 + (i * TPR + t) * 8) * (dt == MOE_F32 ? 4 : 2);
    const Wide8 w = wide_from_f32(v, dt);
    __builtin_amdgcn_raw_buffer_store_b128(w.a, rs, off, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(w.b, rs, dt == MOE_F32 ? off + 16 : kPastEnd, 0, 0);
  };
  struct Row { Wide8 r[NV], x[NV], u[NV], e[NV]; u32x4 st; uint32_t g32, g16; };
  const uint32_t gate_sz = !a.g || !a.gate_token ? 0u : a.gdt == MOE_F32 ? 4u : 2u;
  auto load_row = [&](Row& q, int64_t row) {
    const bool live = row < a.T;
    if (SPLIT)
      q.st = __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(stats + (live ? row : 0), live ? 16u : 0u),
                                                   0, 0, 0);
    const __amdgpu_buffer_rsrc_t rg =
        make_rsrc(static_cast<const char*>(a.g) + (size_t)(live ? row : 0) * gate_sz,
                  live ? gate_sz : 0u);
    // the one of the other size lies past the end as a whole
    q.g32 = __builtin_amdgcn_raw_buffer_load_b32(rg, gate_sz == 4 ? 0 : kPastEnd, 0, 0);
    q.g16 = __builtin_amdgcn_raw_buffer_load_b16(rg, gate_sz == 2 ? 0 : kPastEnd, 0, 0);
    const __amdgpu_buffer_rsrc_t rr = row_of(a.r, a.rdt, row, w_values);
    const __amdgpu_buffer_rsrc_t rx = row_of(a.dx, a.dxdt, row, w_values);
    const __amdgpu_buffer_rsrc_t ru = row_of(a.u, a.udt, row, u_values);
    const __amdgpu_buffer_rsrc_t re = row_of(a.dr, a.rdt, row, a.dr ? (uint32_t)a.D : 0u);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      q.r[i] = load8(rr, a.rdt, i);
      q.x[i] = load8(rx, a.dxdt, i);
      q.u[i] = load8(ru, a.udt, i);
      q.e[i] = load8(re, a.rdt, i);
    }
  };
  // the same number of turns for every row group: the sums hold barriers
  const int64_t step = (int64_t)gridDim.x * R;
  const int64_t first = (int64_t)blockIdx.x * R;
  Row q;
  load_row(q, first + sub);
  __syncthreads();   // the parameters
  int turn = 0;
  for (int64_t row0 = first; row0 < a.T; row0 += step) {
    const int64_t row = row0 + sub;
    const bool live = row < a.T;
    float r[NV][8], dx[NV][8], u[NV][8], d[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      wide_to_f32(q.r[i], a.rdt, r[i]);
      wide_to_f32(q.x[i], a.dxdt, dx[i]);
      wide_to_f32(q.u[i], a.udt, u[i]);
      wide_to_f32(q.e[i], a.rdt, d[i]);
    }
    const u32x4 st = q.st;
    float gt = 1.f;   // a token's gate
    if (gate_sz) {
      gt = a.gdt == MOE_F32 ? __uint_as_float(q.g32)
         : a.gdt == MOE_BF16 ? __uint_as_float(q.g16 << 16)
                             : (float)__builtin_bit_cast(_Float16, (uint16_t)q.g16);
    }
    load_row(q, row0 + step + sub);
    RowStats rs;
    if (SPLIT) {
      rs = {__uint_as_float(st[0]), __uint_as_float(st[1]), __uint_as_float(st[2]),
            __uint_as_float(st[3]), 0.f};
    } else {
      float sum[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // r'^2, t r', u^2, a u (dr', t, r')
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * 8;
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
          float wv[4], pv[4], gv[4];
          params(0, c, h, wv);
          params(1, c, h, pv);
          params(2, c, h, gv);
#pragma unroll
          for (int j = h; j < h + 4; ++j) {
            const float tt = dx[i][j] * wv[j - h];
            const float au = gv[j - h] * pv[j - h] * u[i][j];
            sum[0] = fmaf(r[i][j], r[i][j], sum[0]);
            sum[1] = fmaf(tt, r[i][j], sum[1]);
            sum[2] = fmaf(u[i][j], u[i][j], sum[2]);
            sum[3] = fmaf(au, d[i][j], sum[3]);
            sum[4] = fmaf(au, tt, sum[4]);
            sum[5] = fmaf(au, r[i][j], sum[5]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      // the halves of sh take turns: a row's reads lie between its barrier and
      // the next row's, after which the half is written again
      row_sums<TPR>(sum, sh[turn][sub]);
      turn ^= 1;
      rs = row_stats(a, sum, gt);
      __builtin_amdgcn_raw_buffer_store_b32(
          __float_as_uint(rs.dg), make_rsrc(a.dg_token + (live ? row : 0), live && a.dg_token ? 4u : 0u),
          t == 0 ? 0 : kPastEnd, 0, 0);
    }
    const float inv = rs.inv, m = rs.m, inv_u = rs.inv_u, mp = rs.mp;
    const __amdgpu_buffer_rsrc_t rd = row_of(a.dr_out, a.rdt, row, (uint32_t)a.D);
    const __amdgpu_buffer_rsrc_t ru = row_of(a.du, a.udt, row, u_values);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * 8;
      float o[8];
#pragma unroll
      for (int h = 0; h < 8; h += 4) {
        float wv[4], pv[4], gv[4];
        params(0, c, h, wv);
        params(1, c, h, pv);
        params(2, c, h, gv);
        // the zeros of a row past the last may have an infinite inverse norm
        if (live) {
          if (a.w) {
#pragma unroll
            for (int j = h; j < h + 4; ++j) {
              dw[i][j] = fmaf(dx[i][j], r[i][j] * inv, dw[i][j]);
              d[i][j] += inv * (dx[i][j] * wv[j - h] - r[i][j] * m);
            }
          }
#pragma unroll
          for (int j = h; j < h + 4; ++j) {
            const float v = u[i][j] * inv_u;
            dg[i][j] = fmaf(a.alpha * d[i][j], v * pv[j - h], dg[i][j]);
            const float dz = gt * gv[j - h] * d[i][j];
            dp[i][j] = fmaf(dz, v, dp[i][j]);
            o[j] = a.p ? inv_u * (dz * pv[j - h] - v * mp) : dz;
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      put8(rd, a.rdt, i, d[i]);
      put8(ru, a.udt, i, o);
    }
  }
  // the workgroup's partials: its row groups' sums in order, then one slot
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    float (*const v)[8] = k == 0 ? dw : k == 1 ? dp : dg;
    if (!(k == 0 ? a.w != nullptr : k == 1 ? a.p != nullptr : gate_ch)) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * 8;
      if constexpr (R > 1) {
        __syncthreads();
        if (sub) {
#pragma unroll
          for (int j = 0; j < 8; ++j) fold[(j * (R - 1) + sub - 1) * TPR + t] = v[i][j];
        }
        __syncthreads();
        if (!sub) {
          for (int s = 0; s < R - 1; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += fold[(j * (R - 1) + s) * TPR + t];
        }
      }
      if (c0 + c < a.D && !sub)
        store8(a.part, MOE_F32, ((size_t)k * gridDim.x + blockIdx.x) * a.D + c0 + c, v[i]);
    }
  }
}

// out[c] = the slots' partials of column c, added in a fixed order: 16
// threads take every 16th slot, then their sums in order. blockIdx.y picks
// the vector.
__global__ __launch_bounds__(1024) void norm_columns_kernel(
    const float* __restrict__ part, int slots, int D, float* o0, float* o1, float* o2) {
  __shared__ float sh[16][64];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int l = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + l;
  float s = 0.f;
  if (c < D) {
    const float* p = part + (size_t)blockIdx.y * slots * D + c;
#pragma unroll 4
    for (int k = g; k < slots; k += 16) s += p[(size_t)k * D];
  }
  sh[g][l] = s;
  __syncthreads();
  if (g == 0 && c < D) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) v += sh[k][l];
    out[c] = v;
  }
}

namespace {

// Workgroups of the backward along its rows, each leaving one slot of
// partials: as many as the compute units hold at once, two of 256 threads or
// one of 512. Above 8192 values the columns' two parts, 8192 and the rest,
// double them, and they run in two rounds.
int bwd_slots(int T, int D) {
  const int rows = D <= 2048 ? 4 : D <= 4096 ? 2 : 1;
  const int most = D <= 1024 ? 512 : 256;
  return (int)std::max<int64_t>(1, std::min<int64_t>(((int64_t)T + rows - 1) / rows, most));
}

}  // namespace

// the slots, and four values a row whose sums have a launch of their own
size_t norm_backward_part_floats(int T, int D) {
  return (size_t)3 * bwd_slots(T, D) * D + (D > 8192 ? (size_t)T * 4 : 0);
}

template <int TPR, int R, int NV, bool SPLIT = false>
static void run_norm_backward(const NormBwdArgs& a, int grid, hipStream_t s) {
  constexpr int cols = TPR * NV * 8;
  hipLaunchKernelGGL((norm_backward_kernel<TPR, R, NV, SPLIT>),
                     dim3(grid, SPLIT ? (a.D + cols - 1) / cols : 1), dim3(TPR * R),
                     3 * cols * sizeof(float), s, a,
                     reinterpret_cast<const float4*>(a.part + (size_t)3 * grid * a.D));
}

hipError_t launch_norm_backward(const NormBwdArgs& a, hipStream_t s) {
  const int slots = bwd_slots(a.T, a.D);
  // 16 values a thread where a row has 64 threads for them: fewer threads
  // share a row's sums, with twice the loads in flight each. 8 a thread took
  // 4096 x 2048 f32 in 51 us, not 48; 8192 x 1024 bf16 in 32, not 29; 8192 x
  // 4096 bf16 in 104, not 99.
  if (a.D <= 512) run_norm_backward<64, 4, 1>(a, slots, s);
  else if (a.D <= 1024) run_norm_backward<64, 4, 2>(a, slots, s);
  else if (a.D <= 2048) run_norm_backward<128, 4, 2>(a, slots, s);
  else if (a.D <= 4096) run_norm_backward<256, 2, 2>(a, slots, s);
  else if (a.D <= 8192) run_norm_backward<512, 1, 2>(a, slots, s);
  else {
    if (a.T > 0) {
      hipLaunchKernelGGL(norm_sums_kernel, wide_grid(a.T), dim3(1024), 0, s, a,
                         reinterpret_cast<float4*>(a.part + (size_t)3 * slots * a.D));
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    run_norm_backward<512, 1, 2, true>(a, slots, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_columns_kernel, dim3((a.D + 63) / 64, 3), dim3(1024), 0, s, a.part,
                     slots, a.D, a.dw, a.p ? a.dp : nullptr, a.dg_channel);
  return hipGetLastError();
}

}  // namespace moe
