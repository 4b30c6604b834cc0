// Which kernel multiplies two MXFP4 operands: the one with the least expected time (host only).
//
// Every kernel gives a workgroup a tile of the output and walks K in steps of 256.  Its time is
// taken as a + r (b + c s): r rounds of workgroups over the CUs (in halves where two share a CU),
// s steps in a row (of the K that one wave walks, where waves share K), and a, b, c of the
// configuration, in microseconds, fitted to 3500 measured calls (m from 4 to 4096, ten (n, k) from
// (512, 8192) to (28672, 4096), in HIP graphs; the fits' errors are 5 to 11% rms, and the calls so
// chosen took 1.0% longer than the best configuration of each on average, 20% at most).  What the
// numbers say: few tokens go to the stream kernel, whose waves walk K apart and pull W at the rate
// of memory; long K over few tiles to the wave kernel (m = 256, 4096 x 14336: 16.2 us against 21 on
// tiles); short K and many tiles to the tiled one (m = 512, 4096 x 4096: 11.4 against 12.1; m =
// 1024, 14336 x 4096: 36.8 against 65).  Splitting K over workgroups with a reduction was measured
// too and gained at one shape of fifty (n = 512, k = 8192): it is not built.
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
  double a, b, c;
};

constexpr int kAny = 1 << 30;
constexpr Mx4Config kConfigs[] = {
    {STREAM, 1, 4, 4, 0, 3, 1, 16, false, false, 1.34, 1.11, 0.713},
    {STREAM, 1, 4, 5, 0, 3, 17, 32, false, false, 1.22, 1.09, 1.092},
    {STREAM, 1, 4, 6, 0, 2, 33, 64, false, false, 0.90, 1.89, 0.766},
    {STREAM, 2, 5, 4, 0, 3, 1, 16, true, false, 0.93, 1.59, 1.091},
    {STREAM, 2, 5, 5, 0, 3, 17, 32, true, false, 0.91, 1.61, 1.449},
    {STREAM, 2, 5, 6, 0, 2, 33, 64, true, false, 0.74, 2.30, 1.077},
    {STREAM, 4, 6, 4, 0, 2, 1, 16, true, true, -1.23, 4.51, 0.973},
    {STREAM, 4, 6, 5, 0, 2, 17, 32, true, true, -1.54, 4.80, 1.113},
    {STREAM, 4, 6, 6, 0, 2, 33, 64, true, true, -1.19, 4.88, 1.515},
    {STREAM, 8, 7, 4, 0, 2, 1, 16, true, true, 1.52, 1.52, 1.631},
    {WAVE, 0, 7, 7, 0, 2, 1, kAny, true, true, -1.03, 8.45, 1.991},
    {WAVE, 1, 7, 6, 0, 2, 1, kAny, true, true, 0.59, 4.88, 1.366},
    {WAVE, 2, 6, 7, 0, 2, 1, kAny, true, true, 0.19, 4.99, 1.268},
    {WAVE, 3, 6, 6, 0, 2, 1, kAny, true, true, 1.03, 2.96, 0.821},
    {WAVE, 4, 6, 5, 0, 2, 1, kAny, true, true, 1.53, 2.03, 0.621},
    {WAVE, 5, 5, 6, 0, 2, 1, kAny, false, false, 1.45, 1.94, 0.575},
    {TILED, 0, 8, 8, 0, 0, 1, kAny, true, true, -10.84, 18.95, 1.285},
    {TILED, 1, 8, 7, 0, 0, 1, kAny, true, true, -4.08, 8.77, 0.899},
    {TILED, 2, 7, 7, 1, 0, 1, kAny, true, true, 2.65, 1.09, 0.623},
    {TILED, 3, 7, 6, 1, 0, 1, kAny, true, true, 3.49, 0.13, 0.453},
    {TILED, 4, 6, 7, 1, 0, 1, kAny, false, false, 4.37, -1.04, 0.459},
    {TILED, 5, 6, 6, 1, 0, 1, kAny, false, false, 4.19, -1.05, 0.339},
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t ceil_shift(int64_t a, int log) { return (a + ((int64_t)1 << log) - 1) >> log; }

// SP24_MX4="stream,row blocks", "wave,configuration" or "tiled,configuration" takes that
// configuration where it can run the call (tuning and tests only).
const Mx4Config* forced(const Mx4Args& a, const char* v) {
  char name[8];
  int id;
  if (sscanf(v, "%7[a-z],%d", name, &id) != 2) return nullptr;
  const Kernel k = strcmp(name, "stream") == 0 ? STREAM : strcmp(name, "wave") == 0 ? WAVE : TILED;
  if (k == TILED && strcmp(name, "tiled") != 0) return nullptr;
  for (const Mx4Config& c : kConfigs)
    if (c.kernel == k && c.id == id && a.m >= c.min_m && a.m <= c.max_m &&
        (!a.gated || (a.hq != nullptr ? c.gated_mx4 : c.gated)))
      return &c;
  return nullptr;
}

const Mx4Config& plan(const Mx4Args& a) {
  const char* v = getenv("SP24_MX4");
  if (v != nullptr && v[0] != '\0')
    if (const Mx4Config* c = forced(a, v)) return *c;
  const Mx4Config* best = nullptr;
  double least = 0;
  const int64_t steps = ceil_shift(a.k, kLogStep);
  for (const Mx4Config& c : kConfigs) {
    if (a.m < c.min_m || a.m > c.max_m || (a.gated && !(a.hq != nullptr ? c.gated_mx4 : c.gated))) continue;
    const int64_t tiles = ceil_shift(a.n, a.gated ? c.log_n - 1 : c.log_n) * ceil_shift(a.m, c.log_m);
    const int64_t parts = ceil_shift(tiles << c.log_share, kLogCus);  // rounds, in 1 / share
    const double rounds = parts <= 1 << c.log_share ? 1.0 : (double)parts / (1 << c.log_share);
    const double t = c.a + rounds * (c.b + c.c * (double)ceil_shift(steps, c.log_kw));
    if (best == nullptr || t < least) {
      best = &c;
      least = t;
    }
  }
  return *best;
}

}  // namespace

hipError_t launch_mx4_gemm(const Mx4Args& a, hipStream_t s) {
  const Mx4Config& c = plan(a);
  if (c.kernel == WAVE) return launch_mx4_wave(c.id, a, s);
  if (c.kernel == TILED) return launch_mx4_tiled(c.id, a, s);
  // output columns of a workgroup: an equal share of the rounds that the row blocks need, in
  // fours (n = 14336: 56 columns on every CU 7.35 us, 64 on most of them 7.62)
  const int most = a.gated ? 8 * c.id : 16 * c.id;
  const int64_t rounds = ceil_div(ceil_div(a.n, most), kCus);
  int rows = (int)ceil_div(ceil_div(a.n, rounds * kCus), 4) * 4;
  if (rows < 16) rows = 16;
  if (rows > most) rows = most;
  if (a.hq != nullptr) rows = (rows + 31) / 32 * 32;  // whole blocks of the MXFP4 output
  return launch_mx4_stream(c.id, rows, a, s);
}

}  // namespace sp24
