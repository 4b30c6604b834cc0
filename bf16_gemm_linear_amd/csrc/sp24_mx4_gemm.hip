// Products of MXFP4 operands: Y[m, n] = sum_k X[m, k] W[n, k], and the gated product
// h = silu(X Wg^T) (X Wu^T), on v_mfma_scale_f32_32x32x64_f8f6f4 (the scales enter the
// instruction; fp32 accumulation).
//
// One wave computes 32 rows of W (gated: 32 gate and 32 up rows) by 32 tokens straight
// from global memory.  Operand layout of the instruction for E2M1 codes: lane l holds row
// l % 32 of A (W) or column l % 32 of B (X) and the 32 values (16 bytes, one scale block)
// of half l / 32 of its 64; accumulator register 4g + e is row 8g + 4 (l / 32) + e of
// column l % 32.
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

__device__ __forceinline__ f32x16 mfma32(i32x4 a, i32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  const i32x8 a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

template <bool GATED, bool MX4OUT>
__global__ __launch_bounds__(256) void mx4_gemm_kernel(Mx4Args p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 31, q = lane >> 5;
  const int n0 = blockIdx.x * 32, m0 = (blockIdx.y * 4 + wave) * 32;
  if (m0 >= p.m) return;
  const int wrows = GATED ? 2 * p.n : p.n;
  const int wn = min(n0 + r, p.n - 1), xm = min(m0 + r, p.m - 1);
  const size_t half = (size_t)p.k / 2;
  f32x16 acc[GATED ? 2 : 1];
#pragma unroll
  for (int g = 0; g < (GATED ? 2 : 1); ++g)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[g][e] = 0.f;
  for (int k0 = 0; k0 < p.k; k0 += 64) {
    const int b = k0 / 32 + q;  // block of this lane
    const i32x4 xv = *reinterpret_cast<const i32x4*>(p.x + xm * half + 16 * (size_t)b);
    const uint32_t sx = p.xs[mx4_scale_word(xm, b / 4, p.m, p.k)] >> (8 * (b & 3));
#pragma unroll
    for (int g = 0; g < (GATED ? 2 : 1); ++g) {
      const int row = wn + g * p.n;
      const i32x4 wv = *reinterpret_cast<const i32x4*>(p.w + row * half + 16 * (size_t)b);
      const uint32_t sw = p.ws[mx4_scale_word(row, b / 4, wrows, p.k)] >> (8 * (b & 3));
      acc[g] = mfma32(wv, xv, acc[g], sw & 255u, sx & 255u);
    }
  }
  const int m = m0 + r;
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    if constexpr (GATED) v[e] = silu_mul(acc[0][e], acc[1][e]);
    else v[e] = acc[0][e];
  }
  if constexpr (MX4OUT) {  // n % 128 == 0: the 32 rows are one block of token m
    uint32_t key = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) key = max(key, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    key = max(key, (uint32_t)__shfl_xor((int)key, 32, 64));
    const uint32_t byte = mx4_scale_byte(key >> 23, key == 0);
    if (m >= p.m) return;
    const uint32_t c0 = mx4_codes8(v, byte), c1 = mx4_codes8(v + 8, byte);
    uint16_t* o = reinterpret_cast<uint16_t*>(p.hq + (size_t)m * (p.n / 2) + n0 / 2) + q;
    o[0] = (uint16_t)c0;
    o[2] = (uint16_t)(c0 >> 16);
    o[4] = (uint16_t)c1;
    o[6] = (uint16_t)(c1 >> 16);
    const int b = n0 / 32;
    if (q == 0)
      reinterpret_cast<uint8_t*>(p.hs + mx4_scale_word(m, b / 4, p.m, p.n))[b & 3] = (uint8_t)byte;
  } else {
    if (m >= p.m) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int n = n0 + 8 * (e / 4) + 4 * q + e % 4;
      if (n < p.n) p.y[(size_t)m * p.n + n] = (uint16_t)f32x2_to_bf16x2(v[e], 0.f);
    }
  }
}

}  // namespace

size_t mx4_gemm_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mx4_gemm(const Mx4Args& a, hipStream_t s) {
  const dim3 grid((a.n + 31) / 32, (a.m + 127) / 128);
  if (a.gated && a.hq != nullptr) hipLaunchKernelGGL((mx4_gemm_kernel<true, true>), grid, dim3(256), 0, s, a);
  else if (a.gated) hipLaunchKernelGGL((mx4_gemm_kernel<true, false>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((mx4_gemm_kernel<false, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace sp24
