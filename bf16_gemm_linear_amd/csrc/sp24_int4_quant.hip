// bf16 <-> integer 4-bit codes with a bf16 scale, and if asked for a zero point, per group of a row.
//
//   symmetric:   s = bf16(amax / 7), q = clamp(rne(w / s), -8, 7) + 8
//   zero points: lo = min(0, min w), hi = max(0, max w), s = bf16((hi - lo) / 15),
//                z = clamp(rne(-lo / s), 0, 15), q = clamp(rne(w / s) + z, 0, 15)
// with s = 1 where that is 0, and s = NaN, q = z = 8 for a group with an Inf or a NaN.  A quotient of two
// bf16 values that is not a tie lies further than 2^-17 of it from one, so quotients to fp32 that are exact where
// fp32 holds them give the codes of exact arithmetic.
//
// A lane takes 8 values (a 16-byte load, a 4-byte store), group / 8 lanes a group: one pass, the group's extremes by
// register exchanges.  HBM bounds both ways: 28672 x 8192 by 64 with zero points (598 MB) 115 to 143 us, back 113 to
// 121 (a copy's rate, 5.2 TB/s, gives 116 and 119); 4096 x 14336 by 128 26 and 29.
#include "sp24_fp8.hpp"
#include "sp24_int4.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t f_max(uint32_t a, uint32_t b) {
  return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}
// over the LANES neighbouring lanes of a group
template <int LANES, class F>
__device__ __forceinline__ uint32_t group_fold(uint32_t v, F f) {
  v = fold_lanes<2>(fold_lanes<1>(v, f), f);
  if constexpr (LANES >= 8) v = fold_lanes<4>(v, f);
  if constexpr (LANES >= 16) v = fold_lanes<8>(v, f);
  return v;
}

// bf16 to nearest even; finite and not negative.  Zero becomes 1: the scale of a group of zeros.
__device__ __forceinline__ uint32_t scale_bits(float s) {
  const uint32_t b = f32_to_bf16_rne(s);
  return b == 0 ? 0x3F80u : b;
}

// a / b from r, about 1 / b: one correction with the exact remainder.  What fp32 holds comes out exactly (a tie
// between two codes, say), the rest to its last bit, which does not matter (see above).
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}
// Where neither leaves fp32's normal range.
__device__ __forceinline__ bool plain(float v) { return v > 0x1p-50f && v < 0x1p50f; }

// units of 8 values; units < 2^31 * 32
template <int GROUP, bool ZEROS>
__global__ __launch_bounds__(kThreads) void int4_quant_kernel(const uint16_t* __restrict__ w, int64_t units,
                                                              uint8_t* __restrict__ codes,
                                                              uint16_t* __restrict__ scales,
                                                              uint8_t* __restrict__ zeros) {
  constexpr int LANES = GROUP / 8;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  // a group's lanes are in one wave and all of them are within the units, or none
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
    const u32x4 d = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w) + u);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(d[i] << 16);
      v[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
    }
    const uint32_t key = group_fold<LANES>(key_max8(d), bits_max);  // the largest magnitude's bits
    const bool odd = key >= 0x7F80u;                                // Inf or NaN
    uint32_t sb;
    float neg = 0.0f, z = 8.0f;
    if constexpr (ZEROS) {
      float lo = 0.0f, hi = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
      }
      hi = __uint_as_float(group_fold<LANES>(__float_as_uint(hi), f_max));
      neg = __uint_as_float(group_fold<LANES>(__float_as_uint(-lo), f_max));  // -lo >= 0
      const float range = hi + neg;  // beyond fp32 for the largest values: their halves are not
      if (plain(range)) sb = scale_bits(quotient(range, 15.0f, 1.0f / 15.0f));
      else sb = scale_bits(range < __builtin_inff() ? range / 15.0f : (0.5f * hi + 0.5f * neg) / 7.5f);
    } else {
      const float amax = __uint_as_float(key << 16);
      sb = scale_bits(plain(amax) ? quotient(amax, 7.0f, 1.0f / 7.0f) : amax / 7.0f);
    }
    const float s = __uint_as_float(sb << 16);
    float t[8];
    if (plain(s)) {
      float r = __builtin_amdgcn_rcpf(s);  // to an ulp or two
      r = fmaf(fmaf(-r, s, 1.0f), r, r);
      if constexpr (ZEROS) z = fminf(rintf(quotient(neg, s, r)), 15.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = quotient(v[i], s, r);
    } else {  // the reciprocal or the remainder can leave fp32's range
      if constexpr (ZEROS) z = fminf(rintf(neg / s), 15.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[i] / s;
    }
    uint32_t q = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float c = rintf(t[i]);
      if constexpr (ZEROS) c = fminf(fmaxf(c + z, 0.0f), 15.0f);
      else c = fminf(fmaxf(c, -8.0f), 7.0f) + 8.0f;
      q |= (uint32_t)c << (4 * (i / 2) + 16 * (i % 2));
    }
    if (odd) {
      sb = 0x7FC0u;
      z = 8.0f;
      q = 0x88888888u;
    }
    __builtin_nontemporal_store(q, reinterpret_cast<uint32_t*>(codes) + u);
    if (u % LANES == 0) {
      scales[u / LANES] = (uint16_t)sb;
      if constexpr (ZEROS) zeros[u / LANES] = (uint8_t)z;
    }
  }
}

// (q - z) s: an integer of at most 8 bits times 8 bits is exact in fp32, and rounded once.
__global__ __launch_bounds__(kThreads) void int4_dequant_kernel(const uint8_t* __restrict__ codes,
                                                                const uint16_t* __restrict__ scales,
                                                                const uint8_t* __restrict__ zeros, int64_t units,
                                                                int lanes_log2, uint16_t* __restrict__ out) {
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
    const uint32_t q = reinterpret_cast<const uint32_t*>(codes)[u];
    const int64_t g = u >> lanes_log2;
    const float s = bf16_to_f32(scales[g]), z = zeros == nullptr ? 8.0f : (float)zeros[g];
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = f32x2_to_bf16x2(((float)(q >> (4 * i) & 15u) - z) * s, ((float)(q >> (4 * i + 16) & 15u) - z) * s);
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(out) + u);
  }
}

int blocks_for(int64_t units, int64_t most) {
  const int64_t b = (units + kThreads - 1) / kThreads;
  return (int)(b < most ? b : most);
}
constexpr int64_t kQuantBlocks = 8192, kDequantBlocks = (int64_t)1 << 22;

template <int GROUP>
hipError_t quant(const uint16_t* w, int64_t units, uint8_t* codes, uint16_t* scales, uint8_t* zeros, hipStream_t s) {
  const dim3 grid(blocks_for(units, kQuantBlocks)), block(kThreads);
  if (zeros != nullptr)
    hipLaunchKernelGGL((int4_quant_kernel<GROUP, true>), grid, block, 0, s, w, units, codes, scales, zeros);
  else
    hipLaunchKernelGGL((int4_quant_kernel<GROUP, false>), grid, block, 0, s, w, units, codes, scales, zeros);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_int4(const uint16_t* w, int64_t rows, int64_t cols, int64_t group, uint8_t* codes,
                             uint16_t* scales, uint8_t* zeros, hipStream_t s) {
  const int64_t units = rows * (cols / 8);
  if (group == 32) return quant<32>(w, units, codes, scales, zeros, s);
  if (group == 64) return quant<64>(w, units, codes, scales, zeros, s);
  return quant<128>(w, units, codes, scales, zeros, s);
}

hipError_t launch_dequant_int4(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t rows,
                               int64_t cols, int64_t group, uint16_t* out, hipStream_t s) {
  const int64_t units = rows * (cols / 8);
  hipLaunchKernelGGL(int4_dequant_kernel, dim3(blocks_for(units, kDequantBlocks)), dim3(kThreads), 0, s, codes, scales,
                     zeros, units, group == 32 ? 2 : group == 64 ? 3 : 4, out);
  return hipGetLastError();
}

}  // namespace sp24
