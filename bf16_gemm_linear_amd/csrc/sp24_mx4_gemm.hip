// Which kernel multiplies two MXFP4 operands: the one with the least expected time (host only).
//
// Every kernel gives a workgroup a tile of the output and walks K in steps of 256.  Its time is
// taken as
//   a + r (b + c s) + d f s + e W + g Y,
// r rounds of workgroups over the CUs (in halves where two share a CU) and f the same unrounded
// (a partly filled last round costs less than a whole one: the chip clocks higher and memory is
// freer), s steps in a row (of the K that one wave walks, where waves share K), W the megabytes of
// the weight (memory streams them) and Y the megabytes written; the factors are each
// configuration's, in microseconds, fitted to 29000 measured calls: 4600 shapes (m from 1 to 9000;
// n to 30600 and k to 28672, layers' and any), up to seven configurations each, in HIP graphs.  The
// fits' errors are 4 to 9% rms.  On 980 shapes kept out of a fit the picks took 1.6% longer than
// the best configuration measured, 11% at the 95th percentile (of all: 1.0% from 1025 tokens, 1.3%
// to 16, 2.8% from 65 to 256); with a, b and c alone it was 2.7%.
// What the numbers say (HIP graphs): few tokens go to the stream kernel, whose waves walk K apart and
// pull W at the rate of memory; long K over few tiles to the wave kernel (m = 256, 4096 x 14336: 16.2 us
// against 23.2 on tiles); short K and many tiles to the tiled one (m = 1024, 14336 x 4096: 35.9 against
// 62.8), on 128 x 128 tiles until rounds of 256 x 256 are many or well filled (5000 x 4096 x 4096: 55.2
// us against 61.3; 6000 x 8192 x 8192: 238 against 197).  Near a balance the cards differ (gated 2047 x
// 14336 x 4096: 128 x 128 7 to 10% ahead on one, 3% behind on another).
// Measured and not built: splitting K of the tiled kernel over workgroups with a reduction (gained at one shape of
// fifty, n = 512, k = 8192), and a call's columns in two launches, whole rounds of large tiles and
// the rest on small ones (slower or equal at 12 of 14 shapes).
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

constexpr int kLogCus = 8, kCus = 1 << kLogCus, kLogStep = 8;
enum Kernel { STREAM = 0, WAVE = 1, TILED = 2 };

struct Mx4Config {
  Kernel kernel;
  int id;        // stream: row blocks of 16
  int log_n;     // log2 of a tile's rows of W (gated: gate and up rows together)
  int log_m;     // log2 of its tokens
  int log_share; // log2 of the workgroups that share a CU
  int log_kw;    // log2 of the waves that share K
  int min_m, max_m;
  bool gated, gated_mx4;  // can run those outputs
  double a, b, c, d, e, g;
};

constexpr int kAny = 1 << 30;
constexpr Mx4Config kConfigs[] = {
    {STREAM, 1, 4, 4, 0, 3, 1, 16, false, false, 1.21, 1.05, 0.220, 0.142, 0.070, 5.575},
    {STREAM, 1, 4, 5, 0, 3, 17, 32, false, false, 1.06, 0.90, 0.650, 0.153, 0.027, 3.870},
    {STREAM, 1, 4, 6, 0, 2, 33, 64, false, false, 0.00, 2.01, 0.701, 0.000, 0.000, 3.018},
    {STREAM, 2, 5, 4, 0, 3, 1, 16, true, false, 1.22, 1.32, 0.197, 0.236, 0.088, 2.439},
    {STREAM, 2, 5, 5, 0, 3, 17, 32, true, false, 1.38, 1.34, 0.682, 0.000, 0.092, 0.540},
    {STREAM, 2, 5, 6, 0, 2, 33, 64, true, false, 0.00, 2.83, 0.736, 0.000, 0.068, 1.238},
    {STREAM, 4, 6, 4, 0, 2, 1, 16, true, true, 0.90, 1.93, 0.120, 0.198, 0.100, 1.196},
    {STREAM, 4, 6, 5, 0, 2, 17, 32, true, true, 0.92, 1.89, 0.320, 0.307, 0.081, 1.366},
    {STREAM, 4, 6, 6, 0, 2, 33, 64, true, true, 0.00, 3.68, 0.897, 0.000, 0.094, 0.245},
    {STREAM, 8, 7, 4, 0, 2, 1, 16, true, true, 1.18, 2.16, 0.174, 0.371, 0.109, 0.206},
    {WAVE, 0, 7, 7, 0, 2, 1, kAny, true, true, 0.00, 6.51, 1.605, 0.338, 0.073, 0.238},
    {WAVE, 1, 7, 6, 0, 2, 1, kAny, true, true, 0.00, 4.21, 1.220, 0.000, 0.097, 0.362},
    {WAVE, 2, 6, 7, 0, 2, 1, kAny, true, true, 0.25, 4.40, 1.134, 0.142, 0.063, 0.166},
    {WAVE, 3, 6, 6, 0, 2, 1, kAny, true, true, 0.51, 2.75, 0.645, 0.000, 0.075, 0.430},
    {WAVE, 4, 6, 5, 0, 2, 1, kAny, true, true, 0.66, 2.10, 0.446, 0.000, 0.095, 0.447},
    {WAVE, 5, 5, 6, 0, 2, 1, kAny, false, false, 1.45, 1.25, 0.478, 0.000, 0.059, 0.958},
    {TILED, 0, 8, 8, 0, 0, 1, kAny, true, true, 0.00, 6.30, 1.565, 0.000, 0.054, 0.106},
    {TILED, 1, 8, 7, 0, 0, 1, kAny, true, true, 0.00, 2.50, 1.095, 0.030, 0.068, 0.173},
    {TILED, 2, 7, 7, 1, 0, 1, kAny, true, true, 2.92, 0.66, 0.247, 0.359, 0.059, 0.049},
    {TILED, 3, 7, 6, 1, 0, 1, kAny, true, true, 2.38, 0.87, 0.387, 0.008, 0.057, 0.002},
    {TILED, 4, 6, 7, 1, 0, 1, kAny, false, false, 3.36, 0.00, 0.269, 0.141, 0.030, 0.154},
    {TILED, 5, 6, 6, 1, 0, 1, kAny, false, false, 2.99, 0.00, 0.145, 0.134, 0.039, 0.159},
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t ceil_shift(int64_t a, int log) { return (a + ((int64_t)1 << log) - 1) >> log; }

int64_t tiles_of(const Mx4Config& c, const Mx4Args& a) {
  return ceil_shift(a.n, a.gated ? c.log_n - 1 : c.log_n) * ceil_shift(a.m, c.log_m);
}

// Whether a configuration can run the call: its tokens, its outputs, and a grid of fewer than 2^32
// threads, which HIP refuses to launch more of (a gated product of 2^21 x 2^17 outputs, 146 GB in
// MXFP4, is past it on 128 x 128 tiles and not on 256 x 256).
bool can_run(const Mx4Config& c, const Mx4Args& a) {
  const int threads = c.kernel == TILED ? (c.id == 1 ? 512 : 256) : 64 << c.log_kw;
  return a.m >= c.min_m && a.m <= c.max_m && (!a.gated || (a.hq != nullptr ? c.gated_mx4 : c.gated)) &&
         tiles_of(c, a) * threads < (int64_t)1 << 32;
}

// SP24_MX4="stream,row blocks", "wave,configuration" or "tiled,configuration" takes that
// configuration where it can run the call; with a "!" after it, it and no other: a call that it
// cannot run fails (tuning and tests only).
const Mx4Config* forced(const Mx4Args& a, const char* v, bool* only) {
  char name[8];
  int id;
  *only = v[strlen(v) - 1] == '!';
  if (sscanf(v, "%7[a-z],%d", name, &id) != 2) return nullptr;
  const Kernel k = strcmp(name, "stream") == 0 ? STREAM : strcmp(name, "wave") == 0 ? WAVE : TILED;
  if (k == TILED && strcmp(name, "tiled") != 0) return nullptr;
  for (const Mx4Config& c : kConfigs)
    if (c.kernel == k && c.id == id && can_run(c, a)) return &c;
  return nullptr;
}

const Mx4Config* plan(const Mx4Args& a) {
  const char* v = getenv("SP24_MX4");
  if (v != nullptr && v[0] != '\0') {
    bool only;
    const Mx4Config* const c = forced(a, v, &only);
    if (c != nullptr || only) return c;
  }
  const Mx4Config* best = nullptr;
  double least = 0;
  const int64_t steps = ceil_shift(a.k, kLogStep);
  const double weight = (a.gated ? 2e-6 : 1e-6) * 0.53 * (double)a.n * a.k, written = 2e-6 * (double)a.m * a.n;
  for (const Mx4Config& c : kConfigs) {
    if (!can_run(c, a)) continue;
    const int64_t tiles = tiles_of(c, a);
    const int64_t parts = ceil_shift(tiles << c.log_share, kLogCus);  // rounds, in 1 / share
    const double rounds = parts <= 1 << c.log_share ? 1.0 : (double)parts / (1 << c.log_share);
    const double s = (double)ceil_shift(steps, c.log_kw);
    const double filled = tiles <= kCus ? 1.0 : (double)tiles / kCus;
    const double t = c.a + rounds * (c.b + c.c * s) + c.d * filled * s + c.e * weight + c.g * written;
    if (best == nullptr || t < least) {
      best = &c;
      least = t;
    }
  }
  return best;
}

}  // namespace

hipError_t launch_mx4_gemm(const Mx4Args& a, hipStream_t s) {
  const Mx4Config* const best = plan(a);
  if (best == nullptr) return hipErrorInvalidConfiguration;  // more outputs than any memory holds, or the override
  const Mx4Config& c = *best;
  if (c.kernel == WAVE) return launch_mx4_wave(c.id, a, s);
  if (c.kernel == TILED) return launch_mx4_tiled(c.id, a, s);
  // output columns of a workgroup: an equal share of the rounds that the row blocks need, in
  // fours (n = 14336, k = 4096 in HIP graphs: 56 columns on every CU 7.41 us, 64 on most of them 7.54;
  // 16 tokens 7.42 and 7.62)
  const int most = a.gated ? 8 * c.id : 16 * c.id;
  const int64_t rounds = ceil_div(ceil_div(a.n, most), kCus);
  int rows = (int)ceil_div(ceil_div(a.n, rounds * kCus), 4) * 4;
  if (rows < 16) rows = 16;
  if (rows > most) rows = most;
  if (a.hq != nullptr) rows = (rows + 31) / 32 * 32;  // whole blocks of the MXFP4 output
  return launch_mx4_stream(c.id, rows, a, s);
}

}  // namespace sp24
