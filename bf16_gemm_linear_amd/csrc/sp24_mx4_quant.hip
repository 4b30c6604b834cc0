// bf16 <-> MXFP4: per block of 32 values of a row, e = floor(log2 amax) - 2 clamped to
// [-127, 127] (0 for a block of zeros), codes e2m1_rne(clamp(x 2^-e, +-6)), scale byte
// e + 127; a block with an Inf or NaN gets byte 255 and codes 0.
//
// Memory-bound: 2 + 0.53 bytes a value.  28672 x 8192 takes 103 us, 5.8 TB/s, and 118 to 121 us back,
// 5.0 TB/s, the rate of a large copy (82 with the codes in the last-level cache); 16 x 14336
// takes 2.1 and 1.9 us, of which 1.7 are any launch's.
// A lane takes 8 values (a 16-byte load, a 4-byte store), 4 lanes a block, 16 lanes a word of
// scales.  Non-temporal loads of bf16 and stores of either form: 118 and 119 us without.
#include "sp24_fp8.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

constexpr int kThreads = 256;

// units of 128 values; rows * words < 2^31
__global__ __launch_bounds__(kThreads) void mx4_quant_kernel(const uint16_t* __restrict__ x, uint32_t units,
                                                             uint32_t words, int64_t rows, int64_t cols,
                                                             uint8_t* __restrict__ codes,
                                                             uint32_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63, l16 = threadIdx.x & 15;
  const uint32_t step = gridDim.x * (kThreads / 16);
  for (uint32_t u = blockIdx.x * (kThreads / 16) + threadIdx.x / 16; u < units; u += step) {
    const size_t v = (size_t)u * 16 + l16;
    const u32x4 d = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x) + v);
    const uint32_t byte = mx4_block_byte<7>(key_max8(d));
    __builtin_nontemporal_store(mx4_codes8(d, byte), reinterpret_cast<uint32_t*>(codes) + v);
    const uint32_t word = mx4_word_of_blocks(byte, lane);
    if (l16 == 0) scales[mx4_scale_word(u / words, u % words, rows, cols)] = word;
  }
}

__global__ __launch_bounds__(kThreads) void mx4_dequant_kernel(const uint8_t* __restrict__ codes,
                                                               const uint32_t* __restrict__ scales, uint32_t units,
                                                               uint32_t words, int64_t rows, int64_t cols,
                                                               uint16_t* __restrict__ out) {
  const int l16 = threadIdx.x & 15;
  const uint32_t step = gridDim.x * (kThreads / 16);
  for (uint32_t u = blockIdx.x * (kThreads / 16) + threadIdx.x / 16; u < units; u += step) {
    const size_t v = (size_t)u * 16 + l16;
    const uint32_t q = reinterpret_cast<const uint32_t*>(codes)[v];
    const uint32_t byte = (scales[mx4_scale_word(u / words, u % words, rows, cols)] >> (8 * (l16 >> 2))) & 255u;
    const float s = mx4_scale_f32(byte);
    // E2M1 values are exact in fp32; times a power of two they keep 2 bits, so the
    // upper half of the float is the bf16 value (down to 2^-128, a bf16 subnormal)
    u32x4 o;
    const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0);
    const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
    const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2);
    const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
    o[0] = (__float_as_uint(p0[0] * s) >> 16) | (__float_as_uint(p0[1] * s) & 0xFFFF0000u);
    o[1] = (__float_as_uint(p1[0] * s) >> 16) | (__float_as_uint(p1[1] * s) & 0xFFFF0000u);
    o[2] = (__float_as_uint(p2[0] * s) >> 16) | (__float_as_uint(p2[1] * s) & 0xFFFF0000u);
    o[3] = (__float_as_uint(p3[0] * s) >> 16) | (__float_as_uint(p3[1] * s) & 0xFFFF0000u);
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(out) + v);
  }
}

// Workgroups: at most `most`, each then walking the tensor.  28672 x 8192: the quantiser, which
// reads most, takes 103 us with 8192 of them (2048: 108, one unit a thread: 116), the way back,
// which writes most, 82 with one unit a thread (8192: 100), its codes in the last-level cache.
int blocks_for(uint32_t units, uint32_t most) {
  const uint32_t b = (units + kThreads / 16 - 1) / (kThreads / 16);
  return (int)(b < most ? b : most);
}
constexpr uint32_t kQuantBlocks = 8192, kDequantBlocks = 1u << 22;

}  // namespace

hipError_t launch_quant_mxfp4(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, uint32_t* scales,
                              hipStream_t s) {
  const uint32_t words = (uint32_t)(cols / 128), units = (uint32_t)(rows * words);
  hipLaunchKernelGGL(mx4_quant_kernel, dim3(blocks_for(units, kQuantBlocks)), dim3(kThreads), 0, s, x, units, words,
                     rows, cols, codes, scales);
  return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(const uint8_t* codes, const uint32_t* scales, int64_t rows, int64_t cols,
                                uint16_t* out, hipStream_t s) {
  const uint32_t words = (uint32_t)(cols / 128), units = (uint32_t)(rows * words);
  hipLaunchKernelGGL(mx4_dequant_kernel, dim3(blocks_for(units, kDequantBlocks)), dim3(kThreads), 0, s, codes, scales,
                     units, words, rows, cols, out);
  return hipGetLastError();
}

}  // namespace sp24
