// C entry points of the 8-bit block format and of the norms, and the routed
// layer's launches on MOE_F8B128 weights. Every argument is checked before
// the first launch; every launch goes to the caller's stream.
#include <algorithm>
#include <cmath>

#include "f8_internal.h"

using namespace moe;

namespace {

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

inline bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

inline bool plain_type(int dt) { return dt == MOE_F32 || dt == MOE_BF16 || dt == MOE_F16; }

moe_status launched(hipError_t e, const char* where) {
  if (e == hipSuccess) return MOE_OK;
  return set_error(MOE_EHIP, "%s: %s (%s)", where, hipGetErrorName(e), hipGetErrorString(e));
}

// 256 rows of codes stay below 2 GiB
constexpr int kF8MaxK = 1 << 22;

// The layer's workspace: quantised x, the SwiGLU outputs, the pairs' unweighted outputs, the work lists.
struct F8Layout {
  size_t x8, xs, h8, hs, y, tiles, parts, meta, bytes;
  int cap_tiles, cap_parts;
};

F8Layout f8_layout(const moe_plan_desc& d, int D, int F) {
  F8Layout L{};
  const size_t P = (size_t)d.T * d.k + (size_t)d.n_shared * d.T;
  const int n_exp = d.E + d.n_shared;
  L.cap_tiles = n_exp + (int)(P / kFullBM) + 1;
  L.cap_parts = (int)std::min<size_t>(P, n_exp + P / 16);
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align256(o + bytes); return at; };
  L.x8 = take((size_t)d.T * D);
  L.xs = take((size_t)d.T * (D / 128) * 4);
  // codes, or a decode-shaped call's f32 values
  L.h8 = take(P * F * (d.T <= kDecodeT ? 4 : 1));
  L.hs = take(P * (F / 128) * 4);
  // f32: a rounding of every pair to f16 would weigh as much as y's own
  L.y = take(P * D * 4);
  L.tiles = take((size_t)L.cap_tiles * 8);
  L.parts = take((size_t)L.cap_parts * 16);
  L.meta = take(kF8MetaCount * 4);
  L.bytes = o;
  return L;
}

}  // namespace

size_t moe::f8_layer_bytes(const moe_plan_desc& d, int D, int F) {
  return f8_layout(d, D, F).bytes;
}

// A plan's experts of more rows than this take the tile: its 64-row tiles
// read 256 weight rows once for all rows, where a stream of thin groups reads
// them again for every 16 rows. With 32 (64) instead of 16, 512 uniform tokens
// on 128 experts, top-8, D 2048, F 768 take 231 (279) us, not 179; 4096 skewed
// ones 571 (575), not 547.
constexpr int kF8StreamRows = 16;
// ... in plans of at least so many pairs an expert and more than so many in
// all. Below, the tiles' two launches wait for a few workgroups' walks along
// K: us with tiles / with streams alone at the same D and F: 160 tokens on
// 128 experts (10 pairs an expert) 166 / 144, 224 (14) 166 / 149, 256 (16)
// 172 / 174; 32 tokens on 16 experts (16, 256 pairs) 67 / 41; 512 on 33 (62)
// 69 / 130, 1024 on 8 (256) 93 / 125; 1024 skewed ones, top-1 of 128 (8), 119 /
// 78.
constexpr int kF8TilePairs = 16, kF8TileAll = 256;
// Above so many tokens always: one expert may hold them all.
constexpr int kF8StreamT = 1024;

// 0 quantise x and list the groups, 1 gate/up of thin groups, 2 gate/up tile,
// 3 down of thin groups, 4 down tile, 5 combine
int moe::f8_step_phase(int step) {
  static const int ph[kF8Steps] = {1, 3, 2, 5, 4, 6};
  return ph[step];
}

hipError_t moe::launch_f8_step(const F8Plan& p, const F8Layer& l, int step, hipStream_t s) {
  const moe_plan_desc& d = p.desc;
  const F8Layout L = f8_layout(d, l.D, l.F);
  char* b = l.ws;
  const int64_t P = (int64_t)d.T * d.k + (int64_t)d.n_shared * d.T;
  const int n_exp = d.E + d.n_shared;
  // decode-shaped calls: the plan's own groups, and the strips quantise x and
  // h themselves
  const bool raw = p.decode && f8_strip_raw_fits(d.T, std::max(l.D, l.F));
  const bool tiles = d.T > kF8StreamT ||
      (d.T > kF8StreamRows && P >= (int64_t)kF8TilePairs * n_exp && P > kF8TileAll);
  const bool down = step >= 3;
  // one token: two launches, the second with the pairs' sum
  if (d.T == 1 && !(l.o.flags & MOE_OPT_TILED_DECODE) &&
      f8_one_fits(l.D, l.F, d.k, d.n_shared)) {
    if (step != 1 && step != 3) return hipSuccess;
    const F8OneArgs one{l.x, l.xdt, (const uint8_t*)l.wg, (const uint8_t*)l.wu,
                        (const uint8_t*)l.wd, l.wgs, l.wus, l.wds, p.ids, p.tok2pair,
                        p.offsets, p.w, (float*)(b + L.h8), l.y, l.ydt, l.D, l.F, d.k,
                        d.E, d.n_shared, l.o.swiglu_limit};
    return down ? launch_f8_one_down(one, s) : launch_f8_one_gateup(one, s);
  }
  F8Args g{};
  g.mode = down ? 2 : 1;
  g.K = down ? l.F : l.D;
  g.N = down ? l.D : l.F;
  g.B0 = (const uint8_t*)(down ? l.wd : l.wg);
  g.B0s = down ? l.wds : l.wgs;
  g.B1 = (const uint8_t*)l.wu;
  g.B1s = l.wus;
  g.pair_token = p.pair_token;
  g.offsets = p.offsets;
  g.clamp = l.o.swiglu_limit;
  g.odt = MOE_F32;
  g.adt = MOE_F8B128;
  g.A = (const uint8_t*)(b + (down ? L.h8 : L.x8));
  g.As = (const float*)(b + (down ? L.hs : L.xs));
  g.out = b + (down ? L.y : L.h8);
  g.out_s = (float*)(b + L.hs);
  switch (step) {
    case 0: {
      if (raw) return hipSuccess;
      return launch_f8_prepare({l.x, l.xdt, d.T, l.D, (uint8_t*)(b + L.x8), (float*)(b + L.xs),
                                p.counts, p.offsets, n_exp, tiles ? kF8StreamRows : d.T,
                                (int32_t*)(b + L.parts), (int32_t*)(b + L.tiles),
                                (int32_t*)(b + L.meta)}, s);
    }
    case 1: case 3:
      if (raw) {
        g.A = (const uint8_t*)(down ? b + L.h8 : l.x);
        g.adt = down ? MOE_F32 : l.xdt;
        g.lds_rows = d.T;
        g.list = p.dlist;
        g.groups = p.dmeta + kMetaSk1;
        g.max_groups = (int)std::min<int64_t>(n_exp, P);
        return launch_f8_strip(g, l.ncu, s);
      }
      g.list = (const int32_t*)(b + L.parts);
      g.groups = (const int32_t*)(b + L.meta) + kF8Parts;
      // beside tiles an expert has one part at most
      g.max_groups = tiles ? (int)std::min<int64_t>(P, n_exp) : L.cap_parts;
      return launch_f8_stream(g, s);
    case 2: case 4:
      if (!tiles) return hipSuccess;
      g.list = (const int32_t*)(b + L.tiles);
      g.groups = (const int32_t*)(b + L.meta) + kF8Tiles;
      g.max_groups = L.cap_tiles;
      // gate/up in f32: h becomes codes, and one that an error of its sums
      // moves, moves by a whole step (2^-4 of its value and more); down in
      // f32 where y, the pairs' sum, is not rounded to 16 bits
      return launch_f8_tile(g, !down || l.ydt == MOE_F32, s);
    default:
      return launch_combine(b + L.y, false, p.tok2pair, p.w, p.offsets, d.T,
                            l.D, d.k, d.n_shared, d.E, l.ydt, l.y, s);
  }
}

// How a plain product's rows are cut: strips of 64 rows (false), or row tiles
// of 256, then of 128 or 64 (true; g's tile counts). Each kind's time is
// rounds of the compute units x steps of 128 codes x the microseconds that a
// step of its tile was measured to take (8-bit / f16 sums): 256 rows 2.1 /
// 4.1, 128 rows 1.5 / 1.95, 64 rows 0.87 / 1.25, and a strip launch runs at
// 172 TFLOP/s. Full rounds of 256-row tiles with a tail of smaller ones beat
// a last round that few tiles share: 13312 x 4096 x 4096 takes 3 rounds and
// a tail, not 4.
// us on strips / tiles, bf16 out: 128 x 2048 by 2048 11.0 / 15.6, 517 x 1040
// by 1001 10.4 / 15.5, 300 x 512 by 4096 12.2 / 7.9, 100 x 4096 by 8192 49.6 /
// 29.1.
static bool f8_split(F8Args* g, bool f32, int ncu) {
  if (g->M <= 64) return false;
  const double c256 = f32 ? 4.1 : 2.1, c128 = f32 ? 1.95 : 1.5, c64 = f32 ? 1.25 : 0.87;
  const int64_t nnb = ((int64_t)g->N + 255) / 256, nk = (g->K + 127) / 128;
  auto rounds = [&](int64_t tiles) { return (double)((tiles * nnb + ncu - 1) / ncu); };
  double best = 2.0 * ((g->M + 63) / 64 * 64) * g->N * g->K / 172e6;
  bool tile = false;
  const int64_t all = (g->M + 255) / 256, full = all * nnb / ncu * ncu / nnb;
  for (const int64_t t : {all, std::min(full, g->M / 256), (int64_t)0})
    for (const int tail : {128, 64}) {
      const int64_t rest = std::max<int64_t>(0, g->M - t * 256);
      const int64_t n = (rest + tail - 1) / tail;
      const double us = nk * (rounds(t) * c256 + rounds(n) * (tail == 128 ? c128 : c64));
      if (us < best) {
        best = us;
        tile = true;
        g->tiles256 = (int)t;
        g->tail_rows = tail;
        g->tail_tiles = (int)n;
      }
    }
  return tile;
}

extern "C" {

moe_status moe_quant_f8(const void* x, int32_t dtype, int64_t rows, int32_t K,
                        void* q, float* scales, void* stream) {
  if (!plain_type(dtype))
    return set_error(MOE_EUNSUPPORTED, "dtype %d: f32, bf16 or f16 only", dtype);
  if (rows < 0 || K < 8 || K % 8)
    return set_error(MOE_EINVAL, "rows=%lld must be >= 0 and K=%d a positive multiple of 8",
                     (long long)rows, K);
  if (rows > 0 && (!x || !q || !scales)) return set_error(MOE_EINVAL, "x, q or scales is NULL");
  if (!aligned16(x) || !aligned16(q) || !aligned16(scales))
    return set_error(MOE_EINVAL, "x, q and scales must be 16-byte aligned");
  if (rows > ((int64_t)1 << 31) / (((int64_t)K + 127) / 128) - 1)
    return set_error(MOE_EUNSUPPORTED, "rows=%lld x K=%d hold 2^31 blocks or more",
                     (long long)rows, K);
  if (rows == 0) return MOE_OK;
  return launched(launch_quant_rows(x, dtype, rows, K, q, scales,
                                    reinterpret_cast<hipStream_t>(stream)),
                  "row quantiser");
}

moe_status moe_quant_f8_weights(const void* w, int32_t dtype, int64_t mats,
                                int32_t N, int32_t K, void* q, float* scales,
                                void* stream) {
  if (!plain_type(dtype))
    return set_error(MOE_EUNSUPPORTED, "dtype %d: f32, bf16 or f16 only", dtype);
  if (mats < 0 || N < 0 || K < 8 || K % 8)
    return set_error(MOE_EINVAL, "mats=%lld and N=%d must be >= 0 and K=%d a positive "
                     "multiple of 8", (long long)mats, N, K);
  const bool any = mats > 0 && N > 0;
  if (any && (!w || !q || !scales)) return set_error(MOE_EINVAL, "w, q or scales is NULL");
  if (!aligned16(w) || !aligned16(q) || !aligned16(scales))
    return set_error(MOE_EINVAL, "w, q and scales must be 16-byte aligned");
  if (!any) return MOE_OK;
  const int64_t per = (((int64_t)N + 127) / 128) * (((int64_t)K + 127) / 128);
  if (per >= ((int64_t)1 << 31) || mats > (((int64_t)1 << 31) - 1) / per)
    return set_error(MOE_EUNSUPPORTED, "the weights hold 2^31 blocks or more");
  return launched(launch_quant_weights(w, dtype, mats, N, K, q, scales,
                                       reinterpret_cast<hipStream_t>(stream)),
                  "weight quantiser");
}

moe_status moe_gemm_f8(const void* x, const float* x_scales, const void* w,
                       const float* w_scales, int64_t M, int32_t N, int32_t K,
                       void* out, int32_t out_dtype, void* stream) {
  if (!plain_type(out_dtype))
    return set_error(MOE_EUNSUPPORTED, "output dtype %d: f32, bf16 or f16 only", out_dtype);
  if (M < 0 || N < 0 || K < 16 || K % 16 || K > kF8MaxK)
    return set_error(MOE_EINVAL, "M and N must be >= 0 and K=%d a multiple of 16 in 16..%d",
                     K, kF8MaxK);
  const bool any = M > 0 && N > 0;
  if (any && (!x || !x_scales || !w || !w_scales || !out))
    return set_error(MOE_EINVAL, "x, w, their scales and out must be non-NULL");
  if (!aligned16(x) || !aligned16(x_scales) || !aligned16(w) || !aligned16(w_scales) ||
      !aligned16(out))
    return set_error(MOE_EINVAL, "pointers must be 16-byte aligned");
  if (M > (int64_t)INT32_MAX)
    return set_error(MOE_EUNSUPPORTED, "M=%lld must be below 2^31", (long long)M);
  if (!any) return MOE_OK;
  int ncu;
  const moe_status st = current_cus(&ncu);
  if (st != MOE_OK) return st;
  F8Args g{};
  g.M = M; g.N = N; g.K = K; g.adt = MOE_F8B128;
  g.A = (const uint8_t*)x; g.As = x_scales;
  g.B0 = (const uint8_t*)w; g.B0s = w_scales;
  g.out = out; g.odt = out_dtype;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool f32 = out_dtype == MOE_F32;
  if (f8_split(&g, f32, ncu)) return launched(launch_f8_tile(g, f32, s), "8-bit product");
  return launched(launch_f8_strip(g, ncu, s), "8-bit product");
}

// ---- norms --------------------------------------------------------------------

static moe_status norm_desc_ok(const moe_norm_desc* d) {
  if (!d) return set_error(MOE_EINVAL, "desc is NULL");
  if (d->T < 0 || d->D < 8 || d->D % 8)
    return set_error(MOE_EINVAL, "T=%d must be >= 0 and D=%d a positive multiple of 8", d->T, d->D);
  if (d->D > MOE_NORM_MAX_D)
    return set_error(MOE_EUNSUPPORTED, "D=%d above %d", d->D, MOE_NORM_MAX_D);
  if (!plain_type(d->residual_dtype) || !plain_type(d->block_dtype) ||
      !plain_type(d->weight_dtype) || !plain_type(d->gate_dtype))
    return set_error(MOE_EUNSUPPORTED, "residual, block, weight and gate dtypes: f32, bf16 or f16");
  if (!plain_type(d->x_dtype) && d->x_dtype != MOE_F8B128)
    return set_error(MOE_EUNSUPPORTED, "x dtype %d: f32, bf16, f16 or MOE_F8B128", d->x_dtype);
  if (d->gate_kind < MOE_GATE_NONE || d->gate_kind > MOE_GATE_TOKEN)
    return set_error(MOE_EINVAL, "gate kind %d", d->gate_kind);
  if (!std::isfinite(d->alpha) || !std::isfinite(d->eps) || d->eps < 0.f)
    return set_error(MOE_EINVAL, "alpha must be finite, eps finite and >= 0");
  if (d->flags & ~MOE_NORM_UNIT_OFFSET) return set_error(MOE_EINVAL, "flags %d", d->flags);
  return MOE_OK;
}

moe_status moe_norm_forward(const moe_norm_desc* d, const void* residual,
                            const void* block, const void* post_weight,
                            const void* gate, const void* weight,
                            void* residual_out, void* x, float* x_scales,
                            void* stream) {
  const moe_status st = norm_desc_ok(d);
  if (st != MOE_OK) return st;
  // a tensor of no rows has no pointer: NULL says nothing about it
  if (d->T > 0) {
    if (!block && (post_weight || d->gate_kind != MOE_GATE_NONE))
      return set_error(MOE_EINVAL, "a post-norm or a gate needs a block output");
    if (!block && !weight)
      return set_error(MOE_EINVAL, "neither a block nor a weight: nothing to do");
    if (!residual) return set_error(MOE_EINVAL, "residual is NULL");
    if (block && !residual_out) return set_error(MOE_EINVAL, "residual_out is NULL");
    if (weight && !x) return set_error(MOE_EINVAL, "x is NULL");
    if (weight && d->x_dtype == MOE_F8B128 && !x_scales)
      return set_error(MOE_EINVAL, "x_scales is NULL for 8-bit rows");
    if (d->gate_kind != MOE_GATE_NONE && !gate) return set_error(MOE_EINVAL, "gate is NULL");
  }
  for (const void* p : {residual, block, post_weight, gate, weight, (const void*)residual_out,
                        (const void*)x, (const void*)x_scales})
    if (!aligned16(p)) return set_error(MOE_EINVAL, "pointers must be 16-byte aligned");
  if (d->T == 0) return MOE_OK;
  NormArgs a{};
  a.T = d->T; a.D = d->D; a.nb = (d->D + 127) / 128;
  a.rdt = d->residual_dtype; a.udt = d->block_dtype; a.xdt = d->x_dtype;
  a.wdt = d->weight_dtype; a.gdt = d->gate_dtype;
  a.gate_token = d->gate_kind == MOE_GATE_TOKEN;
  a.unit = (d->flags & MOE_NORM_UNIT_OFFSET) != 0;
  a.alpha = d->alpha; a.eps = d->eps;
  a.r = residual; a.u = block; a.p = post_weight;
  a.g = d->gate_kind == MOE_GATE_NONE ? nullptr : gate;
  a.w = weight;
  a.r_out = residual_out; a.x = x; a.xs = x_scales;
  return launched(launch_norm_forward(a, reinterpret_cast<hipStream_t>(stream)), "norm kernel");
}

size_t moe_norm_backward_workspace_bytes(const moe_norm_desc* d) {
  if (norm_desc_ok(d) != MOE_OK) return 0;
  return align256(norm_backward_part_floats(d->T, d->D) * 4);
}

moe_status moe_norm_backward(const moe_norm_desc* d, const void* residual_out,
                             const void* block, const void* post_weight,
                             const void* gate, const void* weight,
                             const void* dresidual_out, const void* dx,
                             void* dresidual, void* dblock,
                             float* dpost_weight, float* dgate, float* dweight,
                             void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = norm_desc_ok(d);
  if (st != MOE_OK) return st;
  if (d->x_dtype == MOE_F8B128)
    return set_error(MOE_EUNSUPPORTED, "dx is f32, bf16 or f16");
  if ((weight && !dweight) || (post_weight && !dpost_weight) ||
      ((d->gate_kind == MOE_GATE_CHANNEL || (d->gate_kind == MOE_GATE_TOKEN && d->T > 0)) &&
       (!gate || !dgate)))
    return set_error(MOE_EINVAL, "a parameter or its gradient is NULL");
  if (d->T > 0) {   // as in the forward; the parameters' gradients are zeros without rows
    if (!block && (post_weight || d->gate_kind != MOE_GATE_NONE))
      return set_error(MOE_EINVAL, "a post-norm or a gate needs a block output");
    if (!weight && !dresidual_out)
      return set_error(MOE_EINVAL, "neither a weight nor dresidual_out: no gradient comes in");
    if (!dresidual || (block && !dblock) || (weight && (!residual_out || !dx)))
      return set_error(MOE_EINVAL, "residual_out, dx, dresidual or dblock is NULL");
  }
  for (const void* p : {residual_out, block, post_weight, gate, weight, dresidual_out, dx,
                        (const void*)dresidual, (const void*)dblock, (const void*)dpost_weight,
                        (const void*)dgate, (const void*)dweight})
    if (!aligned16(p)) return set_error(MOE_EINVAL, "pointers must be 16-byte aligned");
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return set_error(MOE_EINVAL, "workspace NULL or not 256-byte aligned");
  const size_t need = align256(norm_backward_part_floats(d->T, d->D) * 4);
  if (ws_bytes < need)
    return set_error(MOE_EWORKSPACE, "norm workspace %zu bytes < %zu needed", ws_bytes, need);
  NormBwdArgs a{};
  a.T = d->T; a.D = d->D;
  a.rdt = d->residual_dtype; a.udt = d->block_dtype; a.dxdt = d->x_dtype;
  a.wdt = d->weight_dtype; a.gdt = d->gate_dtype;
  a.gate_token = d->gate_kind == MOE_GATE_TOKEN;
  a.unit = (d->flags & MOE_NORM_UNIT_OFFSET) != 0;
  a.alpha = d->alpha; a.eps = d->eps;
  a.r = residual_out; a.u = block; a.p = post_weight;
  a.g = d->gate_kind == MOE_GATE_NONE ? nullptr : gate;
  a.w = weight;
  a.dr = dresidual_out; a.dx = dx;
  a.dr_out = dresidual; a.du = dblock;
  a.dw = weight ? dweight : nullptr;
  a.dp = post_weight ? dpost_weight : nullptr;
  a.dg_channel = d->gate_kind == MOE_GATE_CHANNEL ? dgate : nullptr;
  a.dg_token = d->gate_kind == MOE_GATE_TOKEN ? dgate : nullptr;
  a.part = static_cast<float*>(ws);
  return launched(launch_norm_backward(a, reinterpret_cast<hipStream_t>(stream)),
                  "norm backward kernel");
}

}  // extern "C"
