// Products with integer 4-bit weights: Y = X W^T, w = (q - z) s with a scale (and zero point) per group.
//
// One wave holds 16 rows of W by 16 rows of X (v_mfma_f32_16x16x32_bf16) and walks K in steps of 32
// values: codes become the bf16 integers q - z, exactly; a group's products are summed in fp32 without
// its scale, which is multiplied in once a group, in fp32: no value of W is ever rounded.
// Lane l holds row l % 16 (A: X, B: W) and values 8 (l / 16) .. + 7 of the step; accumulator register
// e is X row 4 (l / 16) + e, W row l % 16, so a lane has one scale.
#include "sp24_int4.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

enum { PLAIN = 0, GATED = 1, DOWN = 2 };

struct Args {
  int m, n, k, group;  // n: output columns; GATED: W has 2 n rows an expert
  const uint16_t* x;
  Int4Weight w;
  uint16_t* y;  // PLAIN, GATED
  float* part;  // DOWN
  Pairs pairs;  // GATED, DOWN
};

template <int MODE>
__global__ __launch_bounds__(64) void int4_wave_kernel(Args p) {
  const int lane = threadIdx.x, r = lane & 15, q = lane >> 4;
  const int nblocks = (p.n + 15) / 16;
  const int n0 = (int)(blockIdx.x % nblocks) * 16, tile = (int)(blockIdx.x / nblocks);
  int expert = 0, first = tile * 16, rows = min(16, p.m - first);
  if constexpr (MODE != PLAIN)
    if (!find_tile<16>(p.pairs, tile, lane, expert, first, rows)) return;
  const int place = first + min(r, rows - 1);
  size_t xrow = place;
  if constexpr (MODE == GATED) xrow = p.pairs.order[place] / p.pairs.top;
  const uint16_t* x = p.x + xrow * p.k + 8 * q;

  constexpr int WS = MODE == GATED ? 2 : 1;
  const int groups = p.k / p.group;
  const uint8_t* codes[WS];
  size_t srow[WS];
#pragma unroll
  for (int i = 0; i < WS; ++i) {
    const size_t row = (size_t)expert * (WS * p.n) + (size_t)i * p.n + min(n0 + r, p.n - 1);
    codes[i] = p.w.codes + row * (p.k / 2) + 4 * q;
    srow[i] = row * groups;
  }
  f32x4 sum[WS];
#pragma unroll
  for (int i = 0; i < WS; ++i) sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int g = 0; g < groups; ++g) {
#pragma unroll
    for (int i = 0; i < WS; ++i) {
      const float s = bf16_to_f32(p.w.scales[srow[i] + g]);
      const float zp = 128.0f + (p.w.zeros == nullptr ? 8.0f : (float)p.w.zeros[srow[i] + g]);
      f32x4 acc{0.f, 0.f, 0.f, 0.f};
      for (int k = g * p.group; k < (g + 1) * p.group; k += 32) {
        const bf16x8 a = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(x + k));
        const bf16x8 b = int4_values(*reinterpret_cast<const uint32_t*>(codes[i] + k / 2), zp);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[i][e] += s * acc[e];
    }
  }
  if (n0 + r >= p.n) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int row = 4 * q + e;
    if (row >= rows) continue;
    if constexpr (MODE == PLAIN) {
      p.y[(size_t)(first + row) * p.n + n0 + r] = (uint16_t)f32x2_to_bf16x2(sum[0][e], 0.0f);
    } else if constexpr (MODE == GATED) {
      p.y[(size_t)(first + row) * p.n + n0 + r] = (uint16_t)f32x2_to_bf16x2(silu_mul(sum[0][e], sum[1][e]), 0.0f);
    } else {
      p.part[(size_t)p.pairs.order[first + row] * p.n + n0 + r] = sum[0][e];
    }
  }
}

template <int MODE>
hipError_t launch(const Args& a, int64_t tiles, hipStream_t s) {
  const int64_t grid = tiles * ((a.n + 15) / 16);
  if (grid * 64 >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;  // HIP counts threads in 32 bits
  hipLaunchKernelGGL((int4_wave_kernel<MODE>), dim3((uint32_t)grid), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int4_gemm(const Int4Gemm& a, hipStream_t s) {
  return launch<PLAIN>(Args{a.m, a.n, a.k, a.group, a.x, a.w, a.y, nullptr, Pairs{}}, (a.m + 15) / 16, s);
}

hipError_t launch_int4_experts(const Int4Experts& a, hipStream_t s) {
  const int64_t tiles = most_tiles(a.pairs.count, a.pairs.experts, 16);
  const hipError_t e =
      launch<GATED>(Args{0, a.f, a.d, a.group, a.x, a.gu, a.h, nullptr, a.pairs}, tiles, s);
  if (e != hipSuccess) return e;
  return launch<DOWN>(Args{0, a.d, a.f, a.group, a.h, a.down, nullptr, a.part, a.pairs}, tiles, s);
}

}  // namespace sp24
