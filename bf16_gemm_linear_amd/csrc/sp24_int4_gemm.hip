// Which kernel multiplies with integer 4-bit weights.
#include "sp24_int4.hpp"

namespace sp24 {
namespace {

// Row blocks of 16 and output columns of a stream workgroup for n columns (`per` of them a row block).
void stream_shape(int n, int per, bool gated, int mb, int& rb, int& cols) {
  rb = 4;
  while (rb > (gated ? 2 : 1) && (n + per * rb - 1) / (per * rb) < 256) rb /= 2;
  if (mb == 4 && rb > 2) rb = 2;
  cols = per * rb;
}

}  // namespace

hipError_t launch_int4_gemm(const Int4Gemm& a, hipStream_t s) {
  if (a.m <= 2) return launch_int4_vec(a, s);
  if (a.m <= 64) {
    const int mb = a.m <= 16 ? 1 : a.m <= 32 ? 2 : 4;
    int rb, cols;
    stream_shape(a.n, 16, false, mb, rb, cols);
    return launch_int4_stream(rb, mb, cols, a, s);
  }
  return launch_int4_tiled(a.m <= 128 ? 3 : a.m <= 1024 ? 2 : 0, a, s);
}

hipError_t launch_int4_experts(const Int4Experts& a, hipStream_t s) {
  const int64_t each = a.pairs.count / a.pairs.experts;  // pairs of an expert
  if (each <= 32) {
    const int mb = each <= 8 ? 1 : 2;
    const hipError_t e = launch_int4_stream_gated(4, mb, 32, a, s);
    return e != hipSuccess ? e : launch_int4_stream_down(4, mb, 64, a, s);
  }
  const hipError_t e = launch_int4_tiled_gated(2, a, s);
  return e != hipSuccess ? e : launch_int4_tiled_down(2, a, s);
}

}  // namespace sp24
