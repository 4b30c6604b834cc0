// Integer 4-bit weights with a scale per group of a row, the products with them, the router and
// the experts' products: helpers and launchers.
//
// A value is (q - z) s: q in 0..15, s the group's bf16 scale, z its zero point (a byte; 8 where
// there are none).  Eight values of a row share a 32-bit word, value j at bits 4 (j / 2) + 16 (j % 2):
// shifted right by 4 i and masked with 0x000F000F the word holds values 2 i and 2 i + 1 in its
// halves, in the order of two bf16 in a register, and with 0x4300 OR-ed into each half it is the
// bf16 pair (128 + q): two instructions for two values.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sp24.h"
#include "sp24_common.hpp"

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

namespace sp24 {

constexpr uint32_t kInt4Zero = 8;  // the zero point where none are given

// Pair i of a word: the bf16 (128 + q) of values 2 i and 2 i + 1 (exact: bf16 steps by 1 there).
__device__ __forceinline__ uint32_t int4_pair(uint32_t word, int i) {
  return ((word >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
}

// The same pair as q - z, exactly (an integer of at most 8 bits); zp = 128 + z.
__device__ __forceinline__ uint32_t int4_pair(uint32_t word, int i, float zp) {
  const uint32_t p = int4_pair(word, i);
  const float lo = __uint_as_float(p << 16) - zp, hi = __uint_as_float(p & 0xFFFF0000u) - zp;
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);  // both upper halves
}

__device__ __forceinline__ bf16x8 int4_values(uint32_t word, float zp) {
  const u32x4 v{int4_pair(word, 0, zp), int4_pair(word, 1, zp), int4_pair(word, 2, zp), int4_pair(word, 3, zp)};
  return __builtin_bit_cast(bf16x8, v);
}

// sp24_int4_quant.hip
hipError_t launch_quant_int4(const uint16_t* w, int64_t rows, int64_t cols, int64_t group, uint8_t* codes,
                             uint16_t* scales, uint8_t* zeros, hipStream_t s);
hipError_t launch_dequant_int4(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t rows,
                               int64_t cols, int64_t group, uint16_t* out, hipStream_t s);

// A weight [rows, k], or one such for each expert, one after the other.
struct Int4Weight {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;  // or nullptr: 8
};

// The pairs (token, slot) of a call, those of an expert next to each other.
struct Pairs {
  int experts, top;
  int64_t count;       // tokens * top
  const int* offsets;  // [experts + 1]: places of expert e are offsets[e] .. offsets[e + 1] - 1
  const int* order;    // [count] pair at each place; in an expert's range ascending
};

// Y[m, n] = X W^T, bf16 out.
struct Int4Gemm {
  int m, n, k, group;
  const uint16_t* x;
  Int4Weight w;
  uint16_t* y;
};
hipError_t launch_int4_gemm(const Int4Gemm& a, hipStream_t s);

// The experts' products, rows being places: h[place, f] = silu(x Wg^T) (x Wu^T) of the pair's token, in
// bf16; part[pair, d] = h[place] Wd^T, in fp32.
struct Int4Experts {
  int64_t tokens;
  int d, f, group;
  Pairs pairs;
  const uint16_t* x;
  Int4Weight gu, down;  // [experts, 2 f, d] (gate rows first) and [experts, d, f]
  uint16_t* h;
  float* part;
};
hipError_t launch_int4_experts(const Int4Experts& a, hipStream_t s);

// The kernels.  sp24_int4_vec.hip: a few tokens; the experts' block with pairs in their own order, y being
// its output.
hipError_t launch_int4_vec(const Int4Gemm& g, hipStream_t s);
hipError_t launch_int4_vec_experts(const Int4Experts& e, const int32_t* ids, const float* weights, uint16_t* y,
                                   hipStream_t s);
// sp24_int4_stream.hip: rb row blocks of 16, 16 mb tokens and `cols` output columns a workgroup.
hipError_t launch_int4_stream(int rb, int mb, int cols, const Int4Gemm& g, hipStream_t s);
hipError_t launch_int4_stream_gated(int rb, int mb, int cols, const Int4Experts& e, hipStream_t s);
hipError_t launch_int4_stream_down(int rb, int mb, int cols, const Int4Experts& e, hipStream_t s);
// sp24_int4_tiled.hip: configuration cfg.
hipError_t launch_int4_tiled(int cfg, const Int4Gemm& g, hipStream_t s);
hipError_t launch_int4_tiled_gated(int cfg, const Int4Experts& e, hipStream_t s);
hipError_t launch_int4_tiled_down(int cfg, const Int4Experts& e, hipStream_t s);

// sp24_experts.hip: pairs whose id is outside 0 .. experts - 1 get no place and add nothing.
hipError_t launch_sort_pairs(const int32_t* ids, int64_t count, int experts, int* offsets, int* order, hipStream_t s);
hipError_t launch_join_pairs(const float* part, const int32_t* ids, const float* weights, int64_t tokens, int top,
                             int experts, int d, uint16_t* y, hipStream_t s);

// sp24_route.hip
hipError_t launch_route(const sp24_router& r, int64_t tokens, const void* logits, const float* bias, int32_t* ids,
                        float* weights, hipStream_t s);

// The tile of up to BM places that tile number `tile` stands for, all experts' tiles counted one
// after the other; false past the last.  Every lane of the wave gets the same answer.
template <int BM>
__device__ __forceinline__ bool find_tile(const Pairs& p, int tile, int lane, int& expert, int& first, int& rows) {
  int base = 0;
  for (int c = 0; c < p.experts; c += 64) {
    const int e = c + lane;
    const int lo = e < p.experts ? p.offsets[e] : 0, hi = e < p.experts ? p.offsets[e + 1] : 0;
    int upto = (hi - lo + BM - 1) / BM;  // tiles of experts c .. e
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    const uint64_t past = __ballot(tile < base + upto);
    if (past != 0) {
      const int at = __ffsll((unsigned long long)past) - 1;
      const int start = at == 0 ? base : base + __shfl(upto, at - 1);
      expert = c + at;
      first = __shfl(lo, at) + (tile - start) * BM;
      rows = min(BM, __shfl(hi, at) - first);
      return true;
    }
    base += __shfl(upto, 63);
  }
  return false;
}

// A bound of the number of such tiles that needs no look at the ids.
inline int64_t most_tiles(int64_t pairs, int experts, int bm) {
  const int64_t used = pairs < experts ? pairs : experts;  // each has one that is not full
  return (pairs - used) / bm + used;
}

}  // namespace sp24
