// Which kernel multiplies two MXFP4 operands: a rule on the sizes (host only).
//
//   m <= 64: the stream kernel (sp24_mx4_stream.hip); the rows of W are shared over the
//     CUs, so that each streams an equal part.
//   above:   LDS tiles (sp24_mx4_tiled.hip).
#include <stdio.h>
#include <stdlib.h>

#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

constexpr int kCus = 256;
constexpr int kStreamMaxM = 64;
constexpr int kTileN[3] = {256, 128, 128}, kTileM[3] = {256, 128, 64};  // W rows, tokens
constexpr int kStepK = 256;

struct Mx4Plan {
  bool stream;
  int cfg;    // stream: row blocks of 16; tiled: configuration
  int rows;   // stream: output columns per workgroup
  int split;  // tiled: slices of K
};

// SP24_MX4="stream,row blocks,rows" or "tiled,configuration,split" overrides the rule
// where the kernel can run the call (tuning and tests only).
bool plan_override(bool gated, bool mx4_out, Mx4Plan* p) {
  const char* v = getenv("SP24_MX4");
  if (v == nullptr || v[0] == '\0') return false;
  int a, b;
  if (sscanf(v, "stream,%d,%d", &a, &b) == 2) {
    if ((a != 1 && a != 2 && a != 4) || (gated && a == 1) || (mx4_out && (a != 4 || b != 32))) return false;
    if (b < 4 || b % 4 != 0 || b > 16 * (gated ? a / 2 : a)) return false;
    *p = Mx4Plan{true, a, b, 1};
    return true;
  }
  if (sscanf(v, "tiled,%d,%d", &a, &b) == 2) {
    if (a < 0 || a > 2 || b < 1 || b > 64 || (gated && b != 1)) return false;
    *p = Mx4Plan{false, a, 0, b};
    return true;
  }
  return false;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

Mx4Plan plan(int64_t m, int64_t n, int64_t k, bool gated, bool mx4_out) {
  Mx4Plan p{};
  const int steps = ceil_div(k, kStepK);
  if (!plan_override(gated, mx4_out, &p)) {
    if (m <= kStreamMaxM) {
      p.stream = true;
      const int most = gated ? 32 : 64;
      int rows = ceil_div(ceil_div(n, kCus), 4) * 4;
      if (rows > most) rows = ceil_div(ceil_div(n, (int64_t)kCus * ceil_div(rows, most)), 4) * 4;
      rows = rows < 16 ? 16 : rows;
      if (mx4_out) rows = 32;
      const int blocks = ceil_div(rows, 16) * (gated ? 2 : 1);
      p.rows = rows;
      p.cfg = blocks <= 1 ? 1 : blocks <= 2 ? 2 : 4;
      p.split = 1;
    } else {
      const int64_t cols = gated ? 2 * n : n;
      p.split = 1;
      for (p.cfg = 0; p.cfg < 2; ++p.cfg)
        if ((int64_t)ceil_div(cols, kTileN[p.cfg]) * ceil_div(m, kTileM[p.cfg]) >= kCus) break;
      if (!gated) {
        const int64_t tiles = (int64_t)ceil_div(cols, kTileN[p.cfg]) * ceil_div(m, kTileM[p.cfg]);
        while (p.split < 16 && tiles * p.split * 2 <= kCus && steps / (2 * p.split) >= 4) p.split *= 2;
      }
    }
  }
  if (!p.stream && p.split > 1) {  // no empty slice
    if (p.split > steps) p.split = steps;
    p.split = ceil_div(steps, ceil_div(steps, p.split));
  }
  return p;
}

}  // namespace

size_t mx4_gemm_ws_bytes(int64_t m, int64_t n, int64_t k) {
  const Mx4Plan p = plan(m, n, k, false, false);
  return p.stream || p.split <= 1 ? 0 : (size_t)p.split * m * n * sizeof(float);
}

hipError_t launch_mx4_gemm(const Mx4Args& a, hipStream_t s) {
  const Mx4Plan p = plan(a.m, a.n, a.k, a.gated, a.hq != nullptr);
  return p.stream ? launch_mx4_stream(p.cfg, p.rows, a, s) : launch_mx4_tiled(p.cfg, p.split, a, s);
}

}  // namespace sp24
