// C entry points of the MXFP4 operators and the norm (include/sp24.h): argument
// checks, all before the first HIP call, and dispatch.
#include "sp24_checks.hpp"
#include "sp24_mx4.hpp"

using namespace sp24;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 21;  // rows of an operand: one workgroup of up to 1024 threads each
constexpr int64_t kMaxNormK = 65536;            // a row lives in one workgroup's registers

constexpr int64_t kMaxK = (int64_t)1 << 24;     // 32-bit offsets inside a tile of 256 rows

bool mx4_cols(int64_t k) { return k >= 128 && k % 128 == 0 && k <= kMaxK; }
bool mx4_rows(int64_t n) { return n >= 1 && n <= kMaxRows; }

size_t code_bytes(int64_t rows, int64_t cols) { return (size_t)rows * (cols / 2); }
size_t scale_bytes(int64_t rows, int64_t cols) { return (size_t)rows * (cols / 32); }
size_t pad(size_t b) { return (b + 255) / 256 * 256; }

struct Span {
  const void* p;
  size_t bytes;
};

// every output against every input and every other output (NULL spans are skipped)
template <int NI, int NO>
bool any_alias(const Span (&in)[NI], const Span (&out)[NO]) {
  for (int o = 0; o < NO; ++o) {
    if (out[o].p == nullptr || out[o].bytes == 0) continue;
    for (int i = 0; i < NI; ++i)
      if (in[i].p != nullptr && overlaps(out[o].p, out[o].bytes, in[i].p, in[i].bytes)) return true;
    for (int j = o + 1; j < NO; ++j)
      if (out[j].p != nullptr && overlaps(out[o].p, out[o].bytes, out[j].p, out[j].bytes)) return true;
  }
  return false;
}

int quant_checks(const void* wide, int64_t rows, int64_t cols, const void* codes, const void* scales, bool to_codes) {
  if (!wide || !codes || !scales) return SP24_ERR_NULL;
  if (rows < 1 || rows > kMaxDim || !mx4_cols(cols) || rows * (cols / 128) >= ((int64_t)1 << 31))
    return SP24_ERR_SHAPE;
  if (!aligned16(wide) || !aligned16(codes) || !aligned16(scales)) return SP24_ERR_ALIGN;
  const Span w{wide, (size_t)rows * cols * 2}, c{codes, code_bytes(rows, cols)}, s{scales, scale_bytes(rows, cols)};
  const bool bad = to_codes ? any_alias({w}, {c, s}) : any_alias({c, s}, {w});
  return bad ? SP24_ERR_ALIAS : SP24_OK;
}

// Workspace of the feed-forward block: the normed activation and the gated product.
struct FfnWs {
  size_t xq, xs, hq, hs, total;
};
FfnWs ffn_ws(int64_t m, int64_t d, int64_t f) {
  FfnWs w;
  w.xq = 0;
  w.xs = w.xq + pad(code_bytes(m, d));
  w.hq = w.xs + pad(scale_bytes(m, d));
  w.hs = w.hq + pad(code_bytes(m, f));
  w.total = w.hs + pad(scale_bytes(m, f));
  return w;
}

bool ffn_shape(int64_t m, int64_t d, int64_t f) {
  return mx4_rows(m) && mx4_cols(d) && mx4_cols(f) && d <= kMaxNormK && mx4_rows(2 * f) && mx4_rows(d);
}

}  // namespace

extern "C" {

size_t sp24_ffn_mxfp4_workspace_size(int64_t m, int64_t d, int64_t f) {
  return ffn_shape(m, d, f) ? ffn_ws(m, d, f).total : 0;
}

int sp24_quant_mxfp4(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* codes_out, uint8_t* scales_out,
                     void* stream) {
  if (const int st = quant_checks(x_bf16, rows, cols, codes_out, scales_out, true)) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return finish(launch_quant_mxfp4(static_cast<const uint16_t*>(x_bf16), rows, cols, codes_out,
                                   reinterpret_cast<uint32_t*>(scales_out), s), s);
}

int sp24_dequant_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out_bf16,
                       void* stream) {
  if (const int st = quant_checks(out_bf16, rows, cols, codes, scales, false)) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return finish(launch_dequant_mxfp4(codes, reinterpret_cast<const uint32_t*>(scales), rows, cols,
                                     static_cast<uint16_t*>(out_bf16), s), s);
}

int sp24_gemm_mxfp4(int64_t m, int64_t n, int64_t k, const uint8_t* x_codes, const uint8_t* x_scales,
                    const uint8_t* w_codes, const uint8_t* w_scales, void* y_bf16, void* stream) {
  if (!x_codes || !x_scales || !w_codes || !w_scales || !y_bf16) return SP24_ERR_NULL;
  if (!mx4_rows(m) || !mx4_rows(n) || !mx4_cols(k)) return SP24_ERR_SHAPE;
  if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales) ||
      !aligned16(y_bf16))
    return SP24_ERR_ALIGN;
  if (any_alias({{x_codes, code_bytes(m, k)}, {x_scales, scale_bytes(m, k)}, {w_codes, code_bytes(n, k)},
                 {w_scales, scale_bytes(n, k)}},
                {Span{y_bf16, (size_t)m * n * 2}}))
    return SP24_ERR_ALIAS;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const Mx4Args a{(int)m, (int)n, (int)k, false, x_codes, reinterpret_cast<const uint32_t*>(x_scales), w_codes,
                  reinterpret_cast<const uint32_t*>(w_scales), static_cast<uint16_t*>(y_bf16), nullptr, nullptr};
  return finish(launch_mx4_gemm(a, s), s);
}

int sp24_gated_mxfp4(int64_t m, int64_t f, int64_t k, const uint8_t* x_codes, const uint8_t* x_scales,
                     const uint8_t* w_codes, const uint8_t* w_scales, void* h_bf16, uint8_t* h_codes,
                     uint8_t* h_scales, void* stream) {
  if (!x_codes || !x_scales || !w_codes || !w_scales) return SP24_ERR_NULL;
  const bool mx = h_bf16 == nullptr;
  if (!mx && (h_codes != nullptr || h_scales != nullptr)) return SP24_ERR_MODE;
  if (mx && (h_codes == nullptr || h_scales == nullptr)) return SP24_ERR_NULL;
  if (!mx4_rows(m) || f < 1 || !mx4_rows(2 * f) || !mx4_cols(k) || (mx && f % 128 != 0)) return SP24_ERR_SHAPE;
  if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales) ||
      !aligned16(h_bf16) || !aligned16(h_codes) || !aligned16(h_scales))
    return SP24_ERR_ALIGN;
  if (any_alias({{x_codes, code_bytes(m, k)}, {x_scales, scale_bytes(m, k)}, {w_codes, code_bytes(2 * f, k)},
                 {w_scales, scale_bytes(2 * f, k)}},
                {Span{h_bf16, (size_t)m * f * 2}, Span{h_codes, code_bytes(m, f)}, Span{h_scales, scale_bytes(m, f)}}))
    return SP24_ERR_ALIAS;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const Mx4Args a{(int)m, (int)f, (int)k, true, x_codes, reinterpret_cast<const uint32_t*>(x_scales), w_codes,
                  reinterpret_cast<const uint32_t*>(w_scales), static_cast<uint16_t*>(h_bf16), h_codes,
                  reinterpret_cast<uint32_t*>(h_scales)};
  return finish(launch_mx4_gemm(a, s), s);
}

int sp24_rmsnorm(int kind, int64_t m, int64_t k, int64_t group, const void* x_bf16, const void* residual_bf16,
                 void* residual_out_bf16, const void* weight_bf16, float eps, void* out, void* scales_out,
                 void* stream) {
  if (kind < SP24_NORM_BF16 || kind > SP24_NORM_MXFP4) return SP24_ERR_MODE;
  if (!x_bf16 || !weight_bf16 || !out || (kind != SP24_NORM_BF16 && !scales_out)) return SP24_ERR_NULL;
  if ((residual_bf16 == nullptr) != (residual_out_bf16 == nullptr)) return SP24_ERR_NULL;
  if (!(eps > 0.0f) || eps > 3.0e38f) return SP24_ERR_MODE;
  if (!mx4_rows(m) || k < 8 || k % 8 != 0 || k > kMaxNormK) return SP24_ERR_SHAPE;
  if (kind == SP24_NORM_FP8_GROUPS && (group < 8 || group % 8 != 0 || k % group != 0)) return SP24_ERR_SHAPE;
  if (kind == SP24_NORM_MXFP4 && k % 128 != 0) return SP24_ERR_SHAPE;
  if (!aligned16(x_bf16) || !aligned16(residual_bf16) || !aligned16(residual_out_bf16) || !aligned16(weight_bf16) ||
      !aligned16(out))
    return SP24_ERR_ALIGN;
  if (kind == SP24_NORM_MXFP4 ? !aligned16(scales_out) : ((uintptr_t)scales_out & 3u) != 0) return SP24_ERR_ALIGN;
  const size_t wide = (size_t)m * k * 2;
  size_t ob = wide, sb = 0;
  if (kind == SP24_NORM_MXFP4) {
    ob = code_bytes(m, k);
    sb = scale_bytes(m, k);
  } else if (kind != SP24_NORM_BF16) {
    ob = (size_t)m * k;
    sb = (size_t)m * (kind == SP24_NORM_FP8_GROUPS ? k / group : 1) * 4;
  } else {
    scales_out = nullptr;
  }
  // the residual may be updated in place
  const void* other = residual_out_bf16 == residual_bf16 ? nullptr : residual_bf16;
  if (any_alias({{x_bf16, wide}, {weight_bf16, (size_t)k * 2}, {other, wide}},
                {Span{out, ob}, Span{scales_out, sb}, Span{residual_out_bf16, wide}}))
    return SP24_ERR_ALIAS;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const NormArgs a{kind, m, k, kind == SP24_NORM_FP8_GROUPS ? group : k, static_cast<const uint16_t*>(x_bf16),
                   static_cast<const uint16_t*>(residual_bf16), static_cast<uint16_t*>(residual_out_bf16),
                   static_cast<const uint16_t*>(weight_bf16), eps, out, scales_out};
  return finish(launch_rmsnorm(a, s), s);
}

int sp24_ffn_mxfp4(int64_t m, int64_t d, int64_t f, const void* x_bf16, const void* residual_bf16,
                   void* residual_out_bf16, const void* weight_bf16, float eps, const uint8_t* gu_codes,
                   const uint8_t* gu_scales, const uint8_t* down_codes, const uint8_t* down_scales, void* y_bf16,
                   void* ws, size_t ws_bytes, void* stream) {
  if (!x_bf16 || !weight_bf16 || !gu_codes || !gu_scales || !down_codes || !down_scales || !y_bf16)
    return SP24_ERR_NULL;
  if ((residual_bf16 == nullptr) != (residual_out_bf16 == nullptr)) return SP24_ERR_NULL;
  if (!(eps > 0.0f) || eps > 3.0e38f) return SP24_ERR_MODE;
  if (!ffn_shape(m, d, f)) return SP24_ERR_SHAPE;
  if (!aligned16(x_bf16) || !aligned16(residual_bf16) || !aligned16(residual_out_bf16) || !aligned16(weight_bf16) ||
      !aligned16(gu_codes) || !aligned16(gu_scales) || !aligned16(down_codes) || !aligned16(down_scales) ||
      !aligned16(y_bf16))
    return SP24_ERR_ALIGN;
  const FfnWs w = ffn_ws(m, d, f);
  if (ws == nullptr || ws_bytes < w.total) return SP24_ERR_WORKSPACE;
  if (!aligned16(ws)) return SP24_ERR_ALIGN;
  const size_t wide = (size_t)m * d * 2;
  const void* other = residual_out_bf16 == residual_bf16 ? nullptr : residual_bf16;
  if (any_alias({{x_bf16, wide}, {weight_bf16, (size_t)d * 2}, {other, wide}, {gu_codes, code_bytes(2 * f, d)},
                 {gu_scales, scale_bytes(2 * f, d)}, {down_codes, code_bytes(d, f)}, {down_scales, scale_bytes(d, f)}},
                {Span{y_bf16, wide}, Span{residual_out_bf16, wide}, Span{ws, w.total}}))
    return SP24_ERR_ALIAS;
  uint8_t* b = static_cast<uint8_t*>(ws);
  uint32_t *xs = reinterpret_cast<uint32_t*>(b + w.xs), *hs = reinterpret_cast<uint32_t*>(b + w.hs);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = launch_rmsnorm(NormArgs{SP24_NORM_MXFP4, m, d, d, static_cast<const uint16_t*>(x_bf16),
                                         static_cast<const uint16_t*>(residual_bf16),
                                         static_cast<uint16_t*>(residual_out_bf16),
                                         static_cast<const uint16_t*>(weight_bf16), eps, b + w.xq, xs}, s);
  if (e == hipSuccess)
    e = launch_mx4_gemm(Mx4Args{(int)m, (int)f, (int)d, true, b + w.xq, xs, gu_codes,
                                reinterpret_cast<const uint32_t*>(gu_scales), nullptr, b + w.hq, hs}, s);
  if (e == hipSuccess)
    e = launch_mx4_gemm(Mx4Args{(int)m, (int)d, (int)f, false, b + w.hq, hs, down_codes,
                                reinterpret_cast<const uint32_t*>(down_scales), static_cast<uint16_t*>(y_bf16), nullptr,
                                nullptr}, s);
  return finish(e, s);
}

}  // extern "C"
