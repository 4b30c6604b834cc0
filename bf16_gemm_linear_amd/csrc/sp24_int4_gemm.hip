// Which kernel multiplies with integer 4-bit weights, and how: the least of the times that a model expects.
//
// Slab kernel, in microseconds, with W = the workgroups, `steps` = 32 columns x 128 values of a row tile a CU:
//   3 + max(steps t, HBM) + (X + W through L2) / 26 TB/s + 2.2 + slices (0.3 + a slice's sums through memory),
// t = 0.1 for tiles of 16 tokens and 0.14 for 32, steps in whole rounds of W over 256 CUs.
// Tiled kernel: 4 + rounds * steps of 64 values * t, t by tile.  Measured beside it (HIP graphs):
// us and in parentheses expected, eight weights in turn: 16 x 4096 x 14336 14.2 (14.8), 16 x 14336 x 4096 11.9 (11.7),
// 32 17.3 (15.3), 64 x 4096 x 14336 28 (28), 48 x 14336 x 4096 21 to 23 (24.9), 128 33 to 36 (45.6); tiled: 256 x 14336 x
// 4096 57 (55), 2047 x 28672 x 8192 961 to 1000 (1028), where the slab kernel takes 65 and 2330.  Slices with 32-token
// tiles are priced too low and 8 column waves too high: 80 and 96 x 14336 x 4096 are cut in three and take 40 and 42
// to 47 (38 and 39), where uncut with 8 column waves, expected at 43.6 and 43.9, they take 32 and 33.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

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

// The best slab plan and its expected time.
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
        const double compute = steps * (mb == 1 ? 0.1 : 0.14), hbm = (double)n * k / 2 / 5e6;
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
  // alone on a CU 55 us for k = 4096 (160 x 14336 x 4096, where the slab kernel takes 78)
  const double t2 = 4 + (small <= kCus ? 0.8 : up(small, 2 * kCus) * 1.47) * steps;
  cfg = t0 < t2 ? 0 : 1;
  return t0 < t2 ? t0 : t2;
}

enum Kernel { VEC, SLAB, TILED, NONE };

// SP24_INT4="vec", "slab,tokens / 16,waves along the columns,waves along K,slices" or "tiled,configuration" takes that
// kernel and form where it can run the call; with a "!" after it, it and no other: a call that it cannot run fails
// (tuning and tests only).
struct Named {
  Kernel kernel = NONE;
  bool only = false;
  int id = 0, cbs = 0, kp = 0, slices = 1;  // id: tokens / 16 or the tiled configuration
};
Named named() {
  Named r;
  const char* const v = getenv("SP24_INT4");
  if (v == nullptr || v[0] == '\0') return r;
  r.only = v[strlen(v) - 1] == '!';
  char name[8];
  const int parts = sscanf(v, "%7[a-z],%d,%d,%d,%d", name, &r.id, &r.cbs, &r.kp, &r.slices);
  if (parts >= 1 && strcmp(name, "vec") == 0) r.kernel = VEC;
  if (parts == 2 && strcmp(name, "tiled") == 0 && (r.id == 0 || r.id == 1)) r.kernel = TILED;
  if (parts == 5 && strcmp(name, "slab") == 0 && (r.id == 1 || r.id == 2) && r.cbs >= 1 && r.kp >= 1 &&
      r.cbs * r.kp <= 16 && r.slices >= 1 && r.slices <= 8)
    r.kernel = SLAB;
  return r;
}

// A dense product's kernel and form.  No group here: the workspace's size does not depend on it.
struct Plan {
  Kernel kernel;
  SlabPlan slab;
  int tiled;
};
Plan plan(int64_t m, int64_t n, int64_t k) {
  Plan p{m <= 2 ? VEC : TILED, SlabPlan{}, 0};
  const Named f = named();
  if (f.kernel == TILED) return Plan{TILED, SlabPlan{}, f.id};
  if (f.kernel == SLAB)
    return Plan{SLAB, SlabPlan{f.id, f.cbs, f.kp, f.slices == 1 ? (int)k : (int)(up(up(k, f.slices), 128) * 128), 0}, 0};
  if (f.only && (f.kernel != VEC || m > 2)) return Plan{NONE, SlabPlan{}, 0};
  if (p.kernel == VEC) return p;
  const double tiled = tiled_plan(m, n, k, p.tiled);
  if (m <= kSlabTokens && slab_plan(m, n, k, p.slab) <= tiled) p.kernel = SLAB;
  return p;
}

}  // namespace

size_t int4_gemm_workspace(int64_t m, int64_t n, int64_t k) {
  const Plan p = plan(m, n, k);
  return p.kernel == SLAB && p.slab.slice < k ? (size_t)up(k, p.slab.slice) * m * n * 4 : 0;
}

hipError_t launch_int4_gemm(const Int4Gemm& a, float* part, hipStream_t s) {
  Plan p = plan(a.m, a.n, a.k);
  if (p.kernel == VEC) return launch_int4_vec(a, s);
  if (p.kernel == TILED) return launch_int4_tiled(p.tiled, a, s);
  if (p.kernel == NONE) return hipErrorInvalidConfiguration;
  SlabPlan& q = p.slab;
  const int fits = slab_chunk(a.m < 16 * q.mb ? a.m : 16 * q.mb, 32 * q.cbs, a.group);
  q.chunk = q.slice < fits ? q.slice : fits;
  // Several passes over LDS: three waves a SIMD instead of two hide more of their starts.  With two and three,
  // us: 77 x 6144 x 4096 by groups of 32 22.0 and 20.2, 96 x 6144 x 4096 by 64 25.6 and 22.5; in one pass by
  // 128 48 x 14336 x 4096 30.2 and 31.1, 16 x 28672 x 4096 18.5 and 19.5.
  if (q.cbs == 4 && q.chunk < q.slice && named().kernel == NONE) q.kp = 3;
  return launch_int4_slab(q, a, part, s);
}

bool int4_experts_by_pairs(int64_t tokens, int64_t pairs, int64_t experts, int64_t d, int64_t f) {
  const int64_t used = pairs < experts ? pairs : experts;
  const Named by_name = named();
  const bool grids = pairs * f < (int64_t)1 << 25 && tokens * d < (int64_t)1 << 26;  // HIP counts threads in 32 bits
  if (by_name.kernel != NONE) return by_name.kernel == VEC && grids;
  return tokens <= 64 && grids && (double)(pairs - used) * d * f * 1.5 <= 25e6;
}

// An expert product's kernel, by its expected time: `rows` rows of W an expert (gated: gate and up rows), k values.
// An expert with p tiles' rows on average has p + 1/2 tiles, or one, and in between a little more, since the experts'
// shares differ.  Scales that come every 32 values (groups below 128) make the slab kernel's steps 1.35 (tiles of 32)
// to 1.6 times as long; a second round of 256 x 256 tiles takes its time however few they are.  Measured for 64 experts
// of 4096 x 1792, 8 a token, gated and down in us:
//   pairs an expert   slab, tiles of 16   slab, tiles of 32   128 x 128 tiles   256 x 256 tiles
//   8                   132 + 82            162 + 84            237 + 124         296 + 148
//   16                  185 + 105           188 + 108           239 + 126         297 + 151
//   37                  356 + 212           306 + 162           260 + 137         306 + 159
//   75                  655 + 379           508 + 260           322 + 176         337 + 180
//   150                 1192 + 650          932 + 468           493 + 279         455 + 265
//   222                 -                   -                   664 + 367         591 + 338
// A tile's step of 64 values costs a part for W and one for each 64 rows that it multiplies.
struct ExpertsPlan {
  int slab, tiled;  // tokens / 16 of a slab workgroup, or 0 and a tiled configuration
};
ExpertsPlan experts_plan(const Pairs& p, int64_t rows, int64_t k, int group) {
  const double pairs = (double)p.count, used = pairs < p.experts ? pairs : p.experts;
  auto tiles = [&](int bm) {
    const double full = pairs / bm / used, over = full - 0.5;
    return used * 0.5 * (1.5 + full + sqrt(over * over + 0.04));
  };
  const double hbm = used * rows * k / 2 / 5e6;
  double least = 1e30;
  ExpertsPlan best{1, 0};
  for (int mb = 1; mb <= 2; ++mb) {
    const double wg = tiles(16 * mb) * up(rows, 64), few = wg < kCus ? kCus / wg : 1;
    const double compute = tiles(16 * mb) * up(rows, 32) * up(k, 128) / kCus * few *
                           (mb == 1 ? 0.13 * (group == 128 ? 1 : 1.6) : 0.2 * (group == 128 ? 1 : 1.35));
    const double t = 3 + (compute > hbm ? compute : hbm);
    if (t < least) {
      least = t;
      best = ExpertsPlan{mb, 0};
    }
  }
  const double slower = group == 128 ? 1 : group == 64 ? 1.1 : 1.27;  // the sums' rescaling
  const double steps = (double)up(k, 64) * slower;
  const double small = tiles(128) * up(rows, 128), large = tiles(256) * up(rows, 256);
  const double t2 = 4 + (0.55 + 0.46 * tiles(64) / tiles(128)) *
                            (small <= kCus ? 0.7 : small < 2 * kCus ? 1 : small / (2 * kCus)) * steps;
  const double t0 = 4 + (0.98 + 0.33 * tiles(64) / tiles(256)) *
                            (large <= kCus ? 1 : large < 1.6 * kCus ? 1.6 : large / kCus) * steps;
  if (t2 < least) {
    least = t2;
    best = ExpertsPlan{0, 1};
  }
  if (t0 < least) best = ExpertsPlan{0, 0};
  return best;
}

// A slab workgroup of 8 waves: as many columns as leave every CU a workgroup; 64 KB of X, so that two fit a CU.
SlabPlan experts_slab(const ExpertsPlan& e, const Pairs& p, int64_t rows, int64_t k, int most) {
  const int64_t tiles = p.count < p.experts ? p.count : p.experts;
  int cbs = most;
  while (cbs > 2 && tiles * up(rows, 32 * cbs) < kCus) cbs /= 2;
  const int fits = 2048 / e.slab;
  return SlabPlan{e.slab, cbs, 8 / cbs, (int)k, (int)(k < fits ? k : fits)};
}

hipError_t launch_int4_experts(const Int4Experts& a, hipStream_t s) {
  const Named f = named();
  if (f.kernel == TILED || f.kernel == SLAB) {  // both products
    auto slab = [&](int k) { return SlabPlan{f.id, f.cbs, f.kp, k, k < 2048 / f.id ? k : 2048 / f.id}; };
    const hipError_t e = f.kernel == TILED ? launch_int4_tiled_gated(f.id, a, s) : launch_int4_slab_gated(slab(a.d), a, s);
    if (e != hipSuccess) return e;
    return f.kernel == TILED ? launch_int4_tiled_down(f.id, a, s) : launch_int4_slab_down(slab(a.f), a, s);
  }
  if (f.only) return hipErrorInvalidConfiguration;
  const ExpertsPlan g = experts_plan(a.pairs, 2 * (int64_t)a.f, a.d, a.group);
  hipError_t e = g.slab ? launch_int4_slab_gated(experts_slab(g, a.pairs, 2 * (int64_t)a.f, a.d, 4), a, s)
                        : launch_int4_tiled_gated(g.tiled, a, s);
  if (e != hipSuccess) return e;
  const ExpertsPlan d = experts_plan(a.pairs, a.d, a.f, a.group);
  return d.slab ? launch_int4_slab_down(experts_slab(d, a.pairs, a.d, a.f, 8), a, s)
                : launch_int4_tiled_down(d.tiled, a, s);
}

}  // namespace sp24
