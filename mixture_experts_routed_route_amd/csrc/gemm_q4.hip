// Products of up to 16 rows with 4-bit weights on gfx950 (moe_gemm_q4).
#include "rows16.h"
#include "q4_internal.h"

namespace moe {

namespace {

template <class O>
__device__ __forceinline__ void store_out(void* out, size_t at, float v) {
  static_cast<O*>(out)[at] = (O)v;
}

// Up to 16 rows of x against strips of 16 weight rows. Every wave streams its own
// part of a strip against x in LDS, without a barrier; where there are fewer strips
// than waves, up to 16 waves share one's blocks and their sums meet in LDS. K whose
// rows do not fit LDS goes in turns of KL values.
template <class S, class O, int FMT, int NI, int RAGGED>
__global__ __launch_bounds__(64 * kRowWaves) void rows_strip_kernel(RowsArgs a, int KL) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int T = (int)a.M;
  const S* x = (const S*)a.x;
  float* part = (float*)(lds + x_lds_bytes<FMT>(T, KL));   // [waves][NI][64], shared strips
  const int blocks = (a.K + 127) / 128, per = KL / 128;
  const int strips = (int)(((int64_t)a.N + 15) / 16);
  const int split = wave_split(strips, blocks, gridDim.x), share = 1 << split;
  const int mine = wave >> split, q = wave & (share - 1), at_once = kRowWaves >> split;
  const int rounds = (strips + gridDim.x * at_once - 1) / (gridDim.x * at_once);
  for (int r = 0; r < rounds; ++r) {
    // neighbouring workgroups take neighbouring strips
    const int strip = (r * at_once + mine) * gridDim.x + blockIdx.x;
    const bool any = strip < strips;
    floatx4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    const WStrip<FMT> m[1] = {
        weight_strip<FMT, RAGGED>(a.w, a.params, a.N, any ? (int64_t)strip * 16 : 0, a.K)};
    for (int b0 = 0; b0 < blocks; b0 += per) {
      const int n = min(per, blocks - b0);
      const int first = b0 + n * q / share, end = any ? b0 + n * (q + 1) / share : first;
      Stream<S, FMT, NI, 1, RAGGED> st;
      st.start(m, first, end, a.K);
      if (r == 0 || per < blocks) {
        if (r || b0) __syncthreads();   // all waves are done with the turn before
        stage_x<S, FMT>(lds, x, T, b0 * 128, KL, a.K);
        __syncthreads();
      }
      st.run(m, lds, T, KL, b0, first, end, a.K, acc);
    }
    if (split) {
      if (r) __syncthreads();   // the round before has been read
#pragma unroll
      for (int e = 0; e < NI; ++e) part[(wave * NI + e) * 64 + lane] = acc[0][e];
      __syncthreads();
      if (q == 0) add_shared<NI>(part, wave, share, acc[0]);
    }
    if (any && q == 0) {
      const int n = strip * 16 + (lane & 15);
#pragma unroll
      for (int e = 0; e < NI; ++e) {
        const int t = 4 * e + (lane >> 4);
        if (t < T && n < a.N) store_out<O>(a.out, (size_t)t * a.N + n, acc[0][e]);
      }
    }
  }
}

template <class S, class O, int FMT, int RAGGED>
hipError_t strip_launch(const RowsArgs& a, int ncu, hipStream_t s) {
  const int strips = (int)(((int64_t)a.N + 15) / 16);
  const int T = (int)a.M, ni = T <= 4 ? 1 : T <= 8 ? 2 : 4;
  const int gx = strips < ncu ? strips : ncu;
  const size_t part = (size_t)kRowWaves * ni * 256;
  const int KL = lds_turn(x_lds_bytes<FMT>(T, 128), x_lds_bytes<FMT>(T, 256), part, a.K);
  const size_t lds = x_lds_bytes<FMT>(T, KL) + part;
#define MOE_STRIP(NI) \
  hipLaunchKernelGGL((rows_strip_kernel<S, O, FMT, NI, RAGGED>), dim3(gx), dim3(64 * kRowWaves), lds, s, a, KL)
  if (ni == 1) MOE_STRIP(1); else if (ni == 2) MOE_STRIP(2); else MOE_STRIP(4);
#undef MOE_STRIP
  return hipGetLastError();
}

template <class S, class O>
hipError_t by_format(const RowsArgs& a, int ncu, hipStream_t s) {
  const bool whole = a.K % 128 == 0;
  switch (a.fmt) {
    case 0:
      return whole ? strip_launch<S, O, 0, kWhole>(a, ncu, s)
           : a.K % 64 ? strip_launch<S, O, 0, kOdd>(a, ncu, s) : strip_launch<S, O, 0, kWords>(a, ncu, s);
    case 1: return whole ? strip_launch<S, O, 1, kWhole>(a, ncu, s) : strip_launch<S, O, 1, kWords>(a, ncu, s);
    case 2: return whole ? strip_launch<S, O, 2, kWhole>(a, ncu, s) : strip_launch<S, O, 2, kWords>(a, ncu, s);
    default: return hipErrorInvalidValue;
  }
}

template <class S>
hipError_t by_output(const RowsArgs& a, int ncu, hipStream_t s) {
  return a.odt == MOE_F32 ? by_format<S, float>(a, ncu, s)
       : a.odt == MOE_BF16 ? by_format<S, __bf16>(a, ncu, s) : by_format<S, _Float16>(a, ncu, s);
}

}  // namespace

hipError_t launch_rows_product(const RowsArgs& a, int ncu, hipStream_t s) {
  if (a.M < 1 || a.M > 16) return hipErrorInvalidValue;
  if (a.xdt == MOE_F16) return by_output<_Float16>(a, ncu, s);
  if (a.xdt == MOE_BF16) return by_output<__bf16>(a, ncu, s);
  return hipErrorInvalidValue;
}

}  // namespace moe
