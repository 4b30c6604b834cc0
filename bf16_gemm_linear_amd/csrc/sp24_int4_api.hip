// C entry points of the integer 4-bit operators, the router and the experts (include/sp24.h):
// argument checks, all before the first HIP call, and dispatch.
#include "sp24_checks.hpp"
#include "sp24_int4.hpp"

using namespace sp24;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 21;
constexpr int64_t kMaxK = (int64_t)1 << 20;  // 32-bit byte offsets inside a tile of 256 bf16 rows
constexpr int64_t kMaxExperts = 1024, kMaxTop = 64;

bool rows_ok(int64_t n) { return n >= 1 && n <= kMaxRows; }
bool group_ok(int64_t g) { return g == 32 || g == 64 || g == 128; }
bool cols_ok(int64_t k, int64_t group) { return k >= group && k <= kMaxK && k % group == 0; }

size_t code_bytes(int64_t rows, int64_t cols) { return (size_t)rows * (cols / 2); }
size_t scale_bytes(int64_t rows, int64_t cols, int64_t group) { return (size_t)rows * (cols / group) * 2; }

int quant_checks(const void* wide, int64_t rows, int64_t cols, int64_t group, const void* codes, const void* scales,
                 const void* zeros, bool to_codes) {
  if (!wide || !codes || !scales) return SP24_ERR_NULL;
  if (!rows_ok(rows) || !group_ok(group) || !cols_ok(cols, group)) return SP24_ERR_SHAPE;
  if (!aligned16(wide) || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros)) return SP24_ERR_ALIGN;
  const size_t sb = scale_bytes(rows, cols, group);
  const Span w{wide, (size_t)rows * cols * 2}, c{codes, code_bytes(rows, cols)}, s{scales, sb}, z{zeros, sb / 2};
  const bool bad = to_codes ? any_alias({w}, {c, s, z}) : any_alias({c, s, z}, {w});
  return bad ? SP24_ERR_ALIAS : SP24_OK;
}

// Workspace of the experts: the order of the pairs, the gated product and the pairs' outputs.
struct ExpertsWs {
  size_t offsets, order, h, part, total;
};
ExpertsWs experts_ws(int64_t tokens, int64_t d, int64_t f, int64_t experts, int64_t top) {
  const size_t pairs = (size_t)tokens * top;
  ExpertsWs w;
  w.offsets = 0;
  w.order = w.offsets + pad((size_t)(experts + 1) * 4);
  w.h = w.order + pad(pairs * 4);
  w.part = w.h + pad(pairs * f * 2);
  w.total = w.part + pad(pairs * d * 4);
  return w;
}

bool experts_shape(int64_t tokens, int64_t d, int64_t f, int64_t experts, int64_t top) {
  return experts >= 1 && experts <= kMaxExperts && top >= 1 && top <= kMaxTop && rows_ok(tokens) &&
         tokens * top <= kMaxRows && cols_ok(d, 32) && cols_ok(f, 32);
}

}  // namespace

extern "C" {

int sp24_quant_int4(const void* w_bf16, int64_t rows, int64_t cols, int64_t group, uint8_t* codes_out,
                    void* scales_out_bf16, uint8_t* zeros_out, void* stream) {
  if (const int st = quant_checks(w_bf16, rows, cols, group, codes_out, scales_out_bf16, zeros_out, true)) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return finish(launch_quant_int4(static_cast<const uint16_t*>(w_bf16), rows, cols, group, codes_out,
                                  static_cast<uint16_t*>(scales_out_bf16), zeros_out, s), s);
}

int sp24_dequant_int4(const uint8_t* codes, const void* scales_bf16, const uint8_t* zeros, int64_t rows, int64_t cols,
                      int64_t group, void* out_bf16, void* stream) {
  if (const int st = quant_checks(out_bf16, rows, cols, group, codes, scales_bf16, zeros, false)) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return finish(launch_dequant_int4(codes, static_cast<const uint16_t*>(scales_bf16), zeros, rows, cols, group,
                                    static_cast<uint16_t*>(out_bf16), s), s);
}

size_t sp24_gemm_int4_workspace_size(int64_t m, int64_t n, int64_t k) {
  return rows_ok(m) && rows_ok(n) && cols_ok(k, 32) ? int4_gemm_workspace(m, n, k) : 0;
}

int sp24_gemm_int4(int64_t m, int64_t n, int64_t k, int64_t group, const void* x_bf16, const uint8_t* codes,
                   const void* scales_bf16, const uint8_t* zeros, void* y_bf16, void* ws, size_t ws_bytes,
                   void* stream) {
  if (!x_bf16 || !codes || !scales_bf16 || !y_bf16) return SP24_ERR_NULL;
  if (!rows_ok(m) || !rows_ok(n) || !group_ok(group) || !cols_ok(k, group)) return SP24_ERR_SHAPE;
  if (!aligned16(x_bf16) || !aligned16(codes) || !aligned16(scales_bf16) || !aligned16(zeros) || !aligned16(y_bf16))
    return SP24_ERR_ALIGN;
  const size_t need = int4_gemm_workspace(m, n, k);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return SP24_ERR_WORKSPACE;
  if (need > 0 && !aligned16(ws)) return SP24_ERR_ALIGN;
  const size_t sb = scale_bytes(n, k, group);
  if (any_alias({{x_bf16, (size_t)m * k * 2}, {codes, code_bytes(n, k)}, {scales_bf16, sb}, {zeros, sb / 2}},
                {Span{y_bf16, (size_t)m * n * 2}, Span{ws, need}}))
    return SP24_ERR_ALIAS;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const Int4Gemm a{(int)m, (int)n, (int)k, (int)group, static_cast<const uint16_t*>(x_bf16),
                   Int4Weight{codes, static_cast<const uint16_t*>(scales_bf16), zeros}, static_cast<uint16_t*>(y_bf16)};
  return finish(launch_int4_gemm(a, static_cast<float*>(ws), s), s);
}

int sp24_route(const sp24_router* router, int64_t tokens, const void* logits, const float* bias_f32, int32_t* ids_out,
               float* weights_out, void* stream) {
  if (!router || !logits || !ids_out || !weights_out) return SP24_ERR_NULL;
  const sp24_router& r = *router;
  if (r.kind != SP24_ROUTE_SOFTMAX && r.kind != SP24_ROUTE_SIGMOID) return SP24_ERR_MODE;
  if (r.logits_fp32 != 0 && r.logits_fp32 != 1) return SP24_ERR_DTYPE;
  if (!(r.factor - r.factor == 0.0f)) return SP24_ERR_MODE;  // Inf, NaN
  if (r.group_best != 1 && r.group_best != 2) return SP24_ERR_MODE;
  if (!rows_ok(tokens) || r.experts < 1 || r.experts > kMaxExperts || r.groups < 1 || r.groups > 64 ||
      r.experts % r.groups != 0 || r.top_groups < 1 || r.top_groups > r.groups || r.top < 1 || r.top > kMaxTop ||
      r.top > r.top_groups * (r.experts / r.groups) || (r.groups > 1 && r.experts / r.groups < r.group_best))
    return SP24_ERR_SHAPE;
  if (!aligned16(logits) || !aligned16(bias_f32) || !aligned16(ids_out) || !aligned16(weights_out))
    return SP24_ERR_ALIGN;
  const size_t out = (size_t)tokens * r.top * 4;
  if (any_alias({{logits, (size_t)tokens * r.experts * (r.logits_fp32 ? 4 : 2)}, {bias_f32, (size_t)r.experts * 4}},
                {Span{ids_out, out}, Span{weights_out, out}}))
    return SP24_ERR_ALIAS;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return finish(launch_route(r, tokens, logits, bias_f32, ids_out, weights_out, s), s);
}

size_t sp24_experts_int4_workspace_size(int64_t tokens, int64_t d, int64_t f, int64_t experts, int64_t top) {
  return experts_shape(tokens, d, f, experts, top) ? experts_ws(tokens, d, f, experts, top).total : 0;
}

int sp24_experts_int4(const sp24_int4_experts* w, int64_t tokens, int64_t top, const void* x_bf16, const int32_t* ids,
                      const float* weights_f32, void* y_bf16, void* ws, size_t ws_bytes, void* stream) {
  if (!w || !w->gu_codes || !w->gu_scales_bf16 || !w->down_codes || !w->down_scales_bf16 || !x_bf16 || !ids ||
      !weights_f32 || !y_bf16)
    return SP24_ERR_NULL;
  const int64_t E = w->experts, d = w->d, f = w->f;
  if (!group_ok(w->group) || !experts_shape(tokens, d, f, E, top) || d % w->group != 0 || f % w->group != 0)
    return SP24_ERR_SHAPE;
  if (!aligned16(w->gu_codes) || !aligned16(w->gu_scales_bf16) || !aligned16(w->gu_zeros) ||
      !aligned16(w->down_codes) || !aligned16(w->down_scales_bf16) || !aligned16(w->down_zeros) ||
      !aligned16(x_bf16) || !aligned16(ids) || !aligned16(weights_f32) || !aligned16(y_bf16))
    return SP24_ERR_ALIGN;
  const ExpertsWs e = experts_ws(tokens, d, f, E, top);
  if (ws == nullptr || ws_bytes < e.total) return SP24_ERR_WORKSPACE;
  if (!aligned16(ws)) return SP24_ERR_ALIGN;
  const size_t wide = (size_t)tokens * d * 2, few = (size_t)tokens * top * 4;
  const size_t gc = code_bytes(E * 2 * f, d), gs = scale_bytes(E * 2 * f, d, w->group);
  const size_t dc = code_bytes(E * d, f), ds = scale_bytes(E * d, f, w->group);
  if (any_alias({{x_bf16, wide}, {ids, few}, {weights_f32, few}, {w->gu_codes, gc}, {w->gu_scales_bf16, gs},
                 {w->gu_zeros, gs / 2}, {w->down_codes, dc}, {w->down_scales_bf16, ds}, {w->down_zeros, ds / 2}},
                {Span{y_bf16, wide}, Span{ws, e.total}}))
    return SP24_ERR_ALIAS;
  uint8_t* b = static_cast<uint8_t*>(ws);
  int *offsets = reinterpret_cast<int*>(b + e.offsets), *order = reinterpret_cast<int*>(b + e.order);
  float* part = reinterpret_cast<float*>(b + e.part);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const Int4Experts a{tokens, (int)d, (int)f, (int)w->group, Pairs{(int)E, (int)top, tokens * top, offsets, order},
                      static_cast<const uint16_t*>(x_bf16),
                      Int4Weight{w->gu_codes, static_cast<const uint16_t*>(w->gu_scales_bf16), w->gu_zeros},
                      Int4Weight{w->down_codes, static_cast<const uint16_t*>(w->down_scales_bf16), w->down_zeros},
                      reinterpret_cast<uint16_t*>(b + e.h), part};
  uint16_t* const y = static_cast<uint16_t*>(y_bf16);
  if (int4_experts_by_pairs(tokens, tokens * top, E, d, f))
    return finish(launch_int4_vec_experts(a, ids, weights_f32, y, s), s);
  hipError_t st = launch_sort_pairs(ids, tokens * top, (int)E, offsets, order, s);
  if (st == hipSuccess) st = launch_int4_experts(a, s);
  if (st == hipSuccess)
    st = launch_join_pairs(part, ids, weights_f32, tokens, (int)top, (int)E, (int)d, y, s);
  return finish(st, s);
}

}  // extern "C"
