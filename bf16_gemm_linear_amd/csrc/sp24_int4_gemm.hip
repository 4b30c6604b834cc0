// Which kernel multiplies with integer 4-bit weights, and how: the least of the times that a model expects.
//
// Slab kernel, in microseconds, with W = the workgroups, `steps` = 32 columns x 128 values of a row tile a CU:
//   3 + max(steps t, HBM) + (X + W through L2) / 26 TB/s + 2.2 + slices (0.3 + a slice's sums through memory),
// t = 0.09 for tiles of 16 tokens and 0.14 for 32, steps in whole rounds of W over 256 CUs.
// Tiled kernel: 4 + rounds * steps of 64 values * t, t by tile.  Measured beside it (HIP graphs):
//   16 x 4096 x 14336 13.7 (expected 13.7), 16 x 14336 x 4096 11.5 (11.2), 128 x 4096 x 14336 40 (45).
#include "sp24_int4.hpp"

namespace sp24 {
namespace {

constexpr int kCus = 256;
constexpr int kLds = 150 * 1024;  // of 160 KB, for X and the scales of a slab workgroup

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Values of K that a slab workgroup's LDS holds for `rows` tokens and `wrows` rows of W.
int slab_chunk(int rows, int wrows, int group) {
  int c = kLds / (2 * rows) / 128 * 128;
  while (c > 128 && 2 * rows * c + wrows * ((c / group) | 1) * 4 > kLds) c -= 128;
  return c;
}

// The best slab plan and its expected time.  No group here: the workspace's size does not depend on it.
double slab_plan(int64_t m, int64_t n, int64_t k, SlabPlan& best) {
  double least = 1e30;
  for (int mb = 1; mb <= 2; ++mb) {
    const int64_t tiles = up(m, 16 * mb);
    for (int cbs = 2; cbs <= 8; cbs *= 2)
      for (int slices = 1; slices <= 8; ++slices) {
        if (slices > 1 && k / slices < 1024) break;
        const int64_t across = up(n, 32 * cbs), wg = tiles * across * slices;
        const int64_t slice = slices == 1 ? k : up(up(k, slices), 128) * 128;
        const double rounds = (double)up(wg, kCus) * kCus / wg;
        const double steps = (double)tiles * up(n, 32) * up(k, 128) / kCus * rounds;
        const double compute = steps * (mb == 1 ? 0.09 : 0.14), hbm = (double)n * k / 2 / 5e6;
        double t = 3 + (compute > hbm ? compute : hbm) + ((double)across * m * k * 2 + (double)tiles * n * k / 2) / 26e6;
        if (slices > 1) t += 2.2 + slices * (0.3 + (double)m * n * 8 / 8e6);
        if (t < least) {
          least = t;
          best = SlabPlan{mb, cbs, cbs == 2 ? 4 : 2, (int)slice, 0};
        }
      }
  }
  return least;
}

// The tiled configuration and its expected time.
double tiled_plan(int64_t m, int64_t n, int64_t k, int& cfg) {
  const double steps = (double)up(k, 64);
  const int64_t large = up(m, 256) * up(n, 256), small = up(m, 128) * up(n, 128);
  const double t0 = 4 + up(large, kCus) * steps * 2.0;
  const double t2 = 4 + (small <= kCus ? 1.0 : up(small, 2 * kCus) * 1.47) * steps;
  cfg = t0 < t2 ? 0 : 2;
  return t0 < t2 ? t0 : t2;
}

}  // namespace

size_t int4_gemm_workspace(int64_t m, int64_t n, int64_t k) {
  SlabPlan q;
  int cfg;
  if (m <= 2 || m > kSlabTokens || slab_plan(m, n, k, q) > tiled_plan(m, n, k, cfg) || q.slice >= k) return 0;
  return (size_t)up(k, q.slice) * m * n * 4;
}

hipError_t launch_int4_gemm(const Int4Gemm& a, float* part, hipStream_t s) {
  if (a.m <= 2) return launch_int4_vec(a, s);
  int cfg;
  const double tiled = tiled_plan(a.m, a.n, a.k, cfg);
  if (a.m <= kSlabTokens) {
    SlabPlan q;
    if (slab_plan(a.m, a.n, a.k, q) <= tiled) {
      const int fits = slab_chunk(a.m < 16 * q.mb ? a.m : 16 * q.mb, 32 * q.cbs, a.group);
      q.chunk = q.slice < fits ? q.slice : fits;
      return launch_int4_slab(q, a, part, s);
    }
  }
  return launch_int4_tiled(cfg, a, s);
}

bool int4_experts_by_pairs(int64_t tokens, int64_t pairs, int64_t experts, int64_t d, int64_t f) {
  const int64_t used = pairs < experts ? pairs : experts;
  const bool grids = pairs * f < (int64_t)1 << 25 && tokens * d < (int64_t)1 << 26;  // HIP counts threads in 32 bits
  return tokens <= 4 && grids && (double)(pairs - used) * d * f * 1.5 <= 50e6;
}

// Pairs an expert, 64 experts of 4096 x 1792, 8 a token, gated and down in us:
//              slab, tiles of 16   slab, tiles of 32   128 x 128 tiles   256 x 256 tiles
//   8 (64)        126 + 69            161 + 82            394 + 202
//   16 (128)      182 + 95            186 + 106           397 + 208
//   37 (300)      -                   329 + 167           289 + 167         352 + 198
//   75 (600)      -                   571 + 279           349 + 210         376 + 221
//   150 (1200)    -                   1049 + 498          532 + 332         467 + 312
//   222 (1777)    -                   1515 + 691          718 + 445         619 + 407
hipError_t launch_int4_experts(const Int4Experts& a, hipStream_t s) {
  const int64_t each = a.pairs.count / a.pairs.experts;  // pairs of an expert
  if (each <= 28) {
    SlabPlan q;
    q.mb = each <= 12 ? 1 : 2;
    const int fits = 2048 / q.mb;  // 64 KB of X: two workgroups a CU
    q.cbs = 4;
    q.kp = 2;
    q.slice = a.d;
    q.chunk = a.d < fits ? a.d : fits;
    const hipError_t e = launch_int4_slab_gated(q, a, s);
    if (e != hipSuccess) return e;
    q.cbs = 8;
    q.kp = 1;
    q.slice = a.f;
    q.chunk = a.f < fits ? a.f : fits;
    return launch_int4_slab_down(q, a, s);
  }
  const int cfg = each <= 110 ? 2 : 0;
  const hipError_t e = launch_int4_tiled_gated(cfg, a, s);
  return e != hipSuccess ? e : launch_int4_tiled_down(cfg, a, s);
}

}  // namespace sp24
