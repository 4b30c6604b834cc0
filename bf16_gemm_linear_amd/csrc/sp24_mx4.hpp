// MXFP4 (microscaled 4-bit floating point) helpers shared by the quantiser, the
// norm and the products: E2M1 codes with one E8M0 scale per block of 32 values
// along a row (the OCP microscaling format).  A value is e2m1 * 2^(scale - 127).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sp24.h"
#include "sp24_common.hpp"
#include "sp24_internal.hpp"

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

namespace sp24 {

// Scale bytes are kept four to a word (128 values of a row), and the words of a
// [rows, cols] operand in the storage order of the 2:4 metadata words: blocks of 4
// words (512 values), in each block every row's words row after row.
__host__ __device__ inline size_t mx4_scale_word(int64_t r, int64_t word, int64_t rows, int64_t cols) {
  return (size_t)meta_index(r, word, rows, cols / 128);
}

// Scale byte of a block whose largest magnitude has the biased exponent E (of a
// bf16 or fp32 value; `zero`: that magnitude is 0): 2^(E - 127 - 2) puts it into
// [4, 8) times the scale, E2M1's top binade plus what saturates to 6.  A block of
// zeros takes 1; an Inf or NaN takes the NaN byte; below 2^-125 the exponent
// stops at E8M0's least, 2^-127 (subnormal maxima have E = 0 and land there).
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t E, bool zero) {
  if (zero) return 127u;
  if (E == 255u) return 255u;
  return E > 2u ? E - 2u : 0u;
}

// The scale as a float (2^(byte - 127); byte 0 is the subnormal 2^-127; NaN for 255).
__device__ __forceinline__ float mx4_scale_f32(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// 8 values -> 8 codes (value j in bits [4j, 4j + 4)) of v / scale, rounded to
// nearest even and saturated at 6 by the conversion itself.  Blocks with the NaN
// byte get codes 0: every product with them is NaN through the scale.
__device__ __forceinline__ uint32_t mx4_codes8(u32x4 bf16, uint32_t byte) {
  const float s = mx4_scale_f32(byte);
  // copies: a bit cast of a vector's element itself takes element 0 whatever the index
  const uint32_t p0 = bf16[0], p1 = bf16[1], p2 = bf16[2], p3 = bf16[3];
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p0), s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p1), s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p2), s, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p3), s, 3);
  return byte == 255u ? 0u : q;
}

__device__ __forceinline__ uint32_t mx4_codes8(const float* v, uint32_t byte) {
  const float s = mx4_scale_f32(byte);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
  return byte == 255u ? 0u : q;
}

// One step of a butterfly over lanes: f(v, the value of the lane OFF away); for OFF 4 and 8 aligned
// groups of OFF lanes hold one value already (steps 1, 2, 4, ... in turn).  Register exchanges
// throughout, a few cycles each; through LDS (a shuffle) a step takes about a hundred.
template <int OFF, class F>
__device__ __forceinline__ uint32_t fold_lanes(uint32_t v, F f) {
  if constexpr (OFF == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return f((uint32_t)r[0], (uint32_t)r[1]);
  } else if constexpr (OFF == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return f((uint32_t)r[0], (uint32_t)r[1]);
  } else {  // within 16 lanes: swaps in a quad, a half row mirrored, a row mirrored
    constexpr int CTRL = OFF == 1 ? 0xB1 : OFF == 2 ? 0x4E : OFF == 4 ? 0x141 : 0x140;
    return f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
  }
}
__device__ __forceinline__ uint32_t bits_max(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint32_t bits_or(uint32_t a, uint32_t b) { return a | b; }
__device__ __forceinline__ uint32_t bits_sum(uint32_t a, uint32_t b) {
  return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}
template <class F>
__device__ __forceinline__ uint32_t fold_wave(uint32_t v, F f) {
  v = fold_lanes<1>(v, f);
  v = fold_lanes<2>(v, f);
  v = fold_lanes<4>(v, f);
  v = fold_lanes<8>(v, f);
  v = fold_lanes<16>(v, f);
  return fold_lanes<32>(v, f);
}

// The scale byte of each 32-value block held by 4 neighbouring lanes (8 values a
// lane), from each lane's largest magnitude `key` (bits of a bf16 with SHIFT 7,
// of a float with SHIFT 23, sign cleared); and the word of the 4 blocks of 16 lanes.
template <int SHIFT>
__device__ __forceinline__ uint32_t mx4_block_byte(uint32_t key) {
  key = fold_lanes<2>(fold_lanes<1>(key, bits_max), bits_max);
  return mx4_scale_byte(key >> SHIFT, key == 0);
}
__device__ __forceinline__ uint32_t mx4_word_of_blocks(uint32_t byte, int lane) {
  const uint32_t w = byte << (8 * ((lane >> 2) & 3));
  return fold_lanes<8>(fold_lanes<4>(w, bits_or), bits_or);
}

// Two floats -> two bf16, nearest even, NaN kept a NaN.
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// silu(g) u.  exp2's argument rounding costs |g| 2^-24 relative, at most 2^-17
// where silu still has bits in bf16's range of a result; the division is IEEE.
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g / (1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g)) * u;
}

// sp24_mx4_quant.hip
hipError_t launch_quant_mxfp4(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, uint32_t* scales,
                              hipStream_t s);
hipError_t launch_dequant_mxfp4(const uint8_t* codes, const uint32_t* scales, int64_t rows, int64_t cols,
                                uint16_t* out, hipStream_t s);

// sp24_norm.hip
struct NormArgs {
  int kind;  // sp24_norm_kind
  int64_t m, k, group;
  const uint16_t* x;
  const uint16_t* residual;  // or nullptr
  uint16_t* residual_out;    // with residual
  const uint16_t* weight;
  float eps;
  void* out;      // bf16, byte codes, or MXFP4 codes
  void* scales;   // fp32, or MXFP4 scale words
};
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t s);

// sp24_mx4_gemm.hip.  W holds n rows; gated: 2n rows, gate rows first, and the
// output h = silu(X Wg^T) (X Wu^T) of n columns goes to y (bf16), or as MXFP4 to
// hq / hs (n % 128 == 0).
struct Mx4Args {
  int m, n, k;
  bool gated;
  const uint8_t* x;
  const uint32_t* xs;
  const uint8_t* w;
  const uint32_t* ws;
  uint16_t* y;
  uint8_t* hq;
  uint32_t* hs;
};
hipError_t launch_mx4_gemm(const Mx4Args& a, hipStream_t s);
// The three kernels, by configuration (sp24_mx4_stream.hip: rb row blocks of 16 and `rows`
// output columns a workgroup; sp24_mx4_wave.hip; sp24_mx4_tiled.hip).
hipError_t launch_mx4_stream(int rb, int rows, const Mx4Args& a, hipStream_t s);
hipError_t launch_mx4_wave(int cfg, const Mx4Args& a, hipStream_t s);
hipError_t launch_mx4_tiled(int cfg, const Mx4Args& a, hipStream_t s);

}  // namespace sp24
