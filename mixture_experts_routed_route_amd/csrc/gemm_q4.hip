// Products of rows with 4-bit weights on gfx950 (moe_gemm_q4), and, on the same
// kernel, the router's map of a few tokens (16-bit weights).
#include "rows16.h"
#include "q4_internal.h"

namespace moe {

namespace {

template <class O>
__device__ __forceinline__ void store_out(void* out, size_t at, float v) {
  static_cast<O*>(out)[at] = (O)v;
}

// Up to 16 rows of x against strips of 16 weight rows. A workgroup's waves share
// K: wave w holds blocks w, w + waves, .. of x's rows as fragments for all its
// strips, and the waves' sums meet in LDS. K beyond waves * NB blocks goes in
// turns that load x again.
template <class S, class O, int FMT, int NI, int NB, bool RAGGED>
__global__ __launch_bounds__(1024) void rows_strip_kernel(RowsArgs a) {
  extern __shared__ float part[];   // [2][waves][NI][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.y * 16;
  const int T = (int)min<int64_t>(16, a.M - t0);
  const int tok = (lane & 3) * 4 + ((lane >> 2) & 3);   // the token of A's row lane & 15
  const int pieces = a.K / 32, blocks = (a.K + 127) / 128;
  const int turns = (blocks + waves * NB - 1) / (waves * NB);
  const S* xr = (const S*)a.x + (size_t)(t0 + (tok < T ? tok : 0)) * a.K;
  XBlock<S, FMT> xb[NB];
  auto load_x = [&](int turn) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int kb = (turn * NB + i) * waves + wave;
      if (kb < blocks)
        xb[i] = make_xblock<S, FMT>([&](int step) {
          const int k = kb * 128 + step * 32 + (lane >> 4) * 8;
          return tok < T && (!RAGGED || k < a.K) ? ldg16(xr + k) : uint4{0u, 0u, 0u, 0u};
        });
    }
  };
  load_x(0);
  const int strips = (a.N + 15) / 16;
  int turn_of = 0;
  for (int strip = blockIdx.x; strip < strips; strip += gridDim.x) {
    const int n = min(strip * 16 + (lane & 15), a.N - 1);
    const WRow row = weight_row<FMT>(a.w, a.params, (size_t)n, a.K);
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int turn = 0; turn < turns; ++turn) {
      WBlock<FMT> wb[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int kb = (turn * NB + i) * waves + wave;
        if (kb < blocks) wb[i] = load_wblock<FMT, RAGGED>(row, kb, pieces);
      }
      if (turns > 1) load_x(turn);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if ((turn * NB + i) * waves + wave < blocks) block_product<S, FMT, NI>(xb[i], wb[i], acc);
    }
    float* p = part + turn_of * (waves * NI * 64);
#pragma unroll
    for (int e = 0; e < NI; ++e) p[(wave * NI + e) * 64 + lane] = acc[e];
    __syncthreads();
    // the other half of `part` takes the next strip: one barrier a strip
    turn_of ^= 1;
    if (threadIdx.x < 64 * NI) {
      float sum = 0.f;
      for (int w = 0; w < waves; ++w) sum += p[w * NI * 64 + threadIdx.x];
      const int t = 4 * wave + (lane >> 4), c = strip * 16 + (lane & 15);
      if (t < T && c < a.N) store_out<O>(a.out, (size_t)(t0 + t) * a.N + c, sum);
    }
  }
}

template <class S, class O, int FMT, bool RAGGED>
hipError_t strip_launch(const RowsArgs& a, int ncu, hipStream_t s) {
  const int blocks = (a.K + 127) / 128, strips = (a.N + 15) / 16;
  const int waves = blocks <= 4 ? 4 : blocks <= 16 ? 8 : 16;
  const int64_t chunks = (a.M + 15) / 16;
  const int ni = a.M <= 4 ? 1 : a.M <= 8 ? 2 : 4;
  const int gx = strips < 2 * ncu ? strips : 2 * ncu;
  for (int64_t c = 0; c < chunks; c += 32768) {
    RowsArgs b = a;
    b.x = (const S*)a.x + (size_t)c * 16 * a.K;
    b.out = (O*)a.out + (size_t)c * 16 * a.N;
    b.M = a.M - c * 16;
    const dim3 grid(gx, (unsigned)(chunks - c < 32768 ? chunks - c : 32768)), block(64 * waves);
    const size_t lds = (size_t)2 * waves * ni * 256;
#define MOE_STRIP(NI, NB) \
  hipLaunchKernelGGL((rows_strip_kernel<S, O, FMT, NI, NB, RAGGED>), grid, block, lds, s, b)
    if (blocks <= waves) {
      if (ni == 1) MOE_STRIP(1, 1); else if (ni == 2) MOE_STRIP(2, 1); else MOE_STRIP(4, 1);
    } else {
      if (ni == 1) MOE_STRIP(1, 2); else if (ni == 2) MOE_STRIP(2, 2); else MOE_STRIP(4, 2);
    }
#undef MOE_STRIP
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class S, class O>
hipError_t by_format(const RowsArgs& a, int ncu, hipStream_t s) {
  const bool ragged = a.K % 128 != 0;
  switch (a.fmt) {
    case 0: return ragged ? strip_launch<S, O, 0, true>(a, ncu, s) : strip_launch<S, O, 0, false>(a, ncu, s);
    case 1: return ragged ? strip_launch<S, O, 1, true>(a, ncu, s) : strip_launch<S, O, 1, false>(a, ncu, s);
    case 2: return ragged ? strip_launch<S, O, 2, true>(a, ncu, s) : strip_launch<S, O, 2, false>(a, ncu, s);
    default: return hipErrorInvalidValue;
  }
}

template <class S>
hipError_t by_output(const RowsArgs& a, int ncu, hipStream_t s) {
  if (a.fmt < 0) {   // the router's map
    if (a.odt != MOE_F32 || a.K % 128) return hipErrorInvalidValue;
    return strip_launch<S, float, -1, false>(a, ncu, s);
  }
  return a.odt == MOE_F32 ? by_format<S, float>(a, ncu, s)
       : a.odt == MOE_BF16 ? by_format<S, __bf16>(a, ncu, s) : by_format<S, _Float16>(a, ncu, s);
}

}  // namespace

hipError_t launch_rows_product(const RowsArgs& a, int ncu, hipStream_t s) {
  if (a.xdt == MOE_F16) return by_output<_Float16>(a, ncu, s);
  if (a.xdt == MOE_BF16) return by_output<__bf16>(a, ncu, s);
  return hipErrorInvalidValue;
}

}  // namespace moe
