// C entry points of the 4-bit quantiser and of products on 4-bit weights. Every
// argument is checked before the first launch; every launch goes to the
// caller's stream.
#include "f8_internal.h"
#include "q4_internal.h"

using namespace moe;

namespace {

inline bool aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

moe_status launched(hipError_t e, const char* where) {
  if (e == hipSuccess) return MOE_OK;
  return set_error(MOE_EHIP, "%s: %s (%s)", where, hipGetErrorName(e), hipGetErrorString(e));
}

// a row of x stays below 2^31 bytes by far, and so do offsets within a row
constexpr int kQ4MaxK = 1 << 22;
// a launch holds fewer than 2^32 threads along x
constexpr int kQ4MaxN = 1 << 26;

}  // namespace

extern "C" {

moe_status moe_quant_q4_weights(const void* w, int32_t dtype, int32_t w_dtype, int64_t rows,
                                int64_t K, void* data, void* scales, void* stream) {
  const int fmt = q4_fmt(w_dtype);
  if (fmt < 0) return set_error(MOE_EUNSUPPORTED, "dtype %d is not a 4-bit format", w_dtype);
  if (dtype != MOE_F32 && dtype != MOE_BF16 && dtype != MOE_F16)
    return set_error(MOE_EUNSUPPORTED, "dtype %d: f32, bf16 or f16 only", dtype);
  const int G = w_dtype == MOE_Q4A64 ? 64 : 32;
  if (rows < 0 || K <= 0 || K % G)
    return set_error(MOE_EINVAL, "rows=%lld must be >= 0 and K=%lld a positive multiple of %d",
                     (long long)rows, (long long)K, G);
  if (rows > 0 && (!w || !data || !scales))
    return set_error(MOE_EINVAL, "w, data or scales is NULL");
  if (!aligned(w, 16) || !aligned(data, 16) || !aligned(scales, 16))
    return set_error(MOE_EINVAL, "w, data and scales must be 16-byte aligned");
  if (rows > ((int64_t)1 << 40) / K)
    return set_error(MOE_EUNSUPPORTED, "the weights hold more than 2^40 values");
  if (rows == 0) return MOE_OK;
  return launched(launch_quant_q4(w, dtype, fmt, rows, K, data, scales,
                                  reinterpret_cast<hipStream_t>(stream)),
                  "4-bit quantiser");
}

moe_status moe_gemm_q4(const void* x, int32_t x_dtype, moe_weight w, int64_t M, int32_t N,
                       int32_t K, void* out, int32_t out_dtype, void* stream) {
  const int fmt = q4_fmt(w.dtype);
  if (fmt < 0) return set_error(MOE_EUNSUPPORTED, "weight dtype %d is not a 4-bit format", w.dtype);
  if (x_dtype != MOE_BF16 && x_dtype != MOE_F16)
    return set_error(MOE_EUNSUPPORTED, "x dtype %d: bf16 or f16 only", x_dtype);
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16 && out_dtype != MOE_F16)
    return set_error(MOE_EUNSUPPORTED, "output dtype %d: f32, bf16 or f16 only", out_dtype);
  const int G = w.dtype == MOE_Q4A64 ? 64 : 32;
  if (M < 0 || N < 0 || K < G || K % G || K > kQ4MaxK)
    return set_error(MOE_EINVAL, "M and N must be >= 0 and K=%d a multiple of %d in %d..%d", K, G, G,
                     kQ4MaxK);
  const bool any = M > 0 && N > 0;
  if (any && (!x || !w.data || !w.scales || !out))
    return set_error(MOE_EINVAL, "x, w, its scales and out must be non-NULL");
  if (!aligned(x, 16) || !aligned(w.data, 16) || !aligned(w.scales, 16) || !aligned(out, 16))
    return set_error(MOE_EINVAL, "pointers must be 16-byte aligned");
  if (M > (int64_t)INT32_MAX || N > kQ4MaxN)
    return set_error(MOE_EUNSUPPORTED, "M=%lld must be below 2^31, N=%d at most 2^26",
                     (long long)M, N);
  if (!any) return MOE_OK;
  int ncu;
  const moe_status st = current_cus(&ncu);
  if (st != MOE_OK) return st;
  const RowsArgs a{x, x_dtype, w.data, w.scales, fmt, M, N, K, out, out_dtype};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return launched(M <= 16 ? launch_rows_product(a, ncu, s) : launch_q4_tile(a, ncu, s),
                  "4-bit product");
}

}  // extern "C"
