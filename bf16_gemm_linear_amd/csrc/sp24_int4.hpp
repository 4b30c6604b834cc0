// Integer 4-bit weights with a scale per group of a row, the products with them, the router and
// the experts' products: helpers and launchers.
//
// A value is (q - z) s: q in 0..15, s the group's bf16 scale, z its zero point (a byte; 8 where
// there are none).  Eight values of a row share a 32-bit word, value j at bits 4 (j / 2) + 16 (j % 2):
// shifted right by 4 i and masked with 0x000F000F the word holds values 2 i and 2 i + 1 in its
// halves, in the order of two bf16 in a register, and with 0x4300 OR-ed into each half it is the
// bf16 pair (128 + q): two instructions for two values.
//
// The kernels for few tokens sum x (c + q - z) and take the sum of c x off behind: c = 136 without zero points,
// where c + q - z is 128 + q, and 192 with them (bf16 from 128 to 255 are integers, one apart).  Both sums are formed by the same instructions in the same order, so where q = z in a
// whole group they are equal bit for bit and the group adds exactly nothing, whatever its scale (the quantiser's
// is 1 for a group of zeros, hundreds of times its neighbours').  Taking (128 + z) times the sum of x off instead
// leaves what the roundings differ by: up to 1e-3 in a row of zeros, beside outputs of about 1.  To subtract z
// from every code before the product takes 21 instructions for 8 values and one token instead of 11 (13 with zero
// points): one token of 14336 x 4096 9.2 us from 8.3 in a graph, 77 x 6144 x 4096 by 32 25 from 21.5.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sp24.h"
#include "sp24_common.hpp"

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

namespace sp24 {

constexpr uint32_t kInt4Zero = 8;  // the zero point where none are given

// Words into pairs of bf16, c + q - z.
template <bool Z>  // with zero points
struct Int4Bits {
  static constexpr uint32_t kConstant = Z ? 0x43404340u : 0x43084308u;  // c, c
  // Constants where one instruction takes two: a vector instruction here has room for one scalar register and no
  // literal, so left to itself the compiler masks and sets in two.
  uint32_t mask, magic;
  __device__ __forceinline__ Int4Bits() : mask(Z ? 0x0F0F0F0Fu : 0x000F000Fu), magic(0x43004300u) {
    asm("" : "+s"(mask));
    asm("" : "+v"(magic));
  }
  // z: Int4Zeros::bytes
  __device__ __forceinline__ bf16x8 values(uint32_t word, uint32_t z) const {
    u32x4 r;
    if constexpr (Z) {
      // 64 + q - z in the bytes: of values 0 4 1 5 and 2 6 3 7; beside 0x43 each is the bf16 192 + q - z
      const uint32_t e = (word & mask) + z, o = (word >> 4 & mask) + z;
      r = u32x4{__builtin_amdgcn_perm(e, magic, 0x01060104u), __builtin_amdgcn_perm(o, magic, 0x01060104u),
                __builtin_amdgcn_perm(e, magic, 0x01070105u), __builtin_amdgcn_perm(o, magic, 0x01070105u)};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = (word >> (4 * i) & mask) | magic;
    }
    return __builtin_bit_cast(bf16x8, r);
  }
};

// A zero point as the kernels use it, in 16 bits: z = part + 3 left, part at most 63, as bytes 64 - part and left.
// 3 / 192 is 1 / 64, so the sum of c x taken off 1 + left / 64 times makes up for the rest, without a rounding of its
// own; left is 0 up to 63.
struct Int4Zeros {
  static __device__ __forceinline__ uint32_t of(uint32_t z) {
    const uint32_t left = z < 64 ? 0 : (z - 61) / 3;
    return left << 8 | (64 - (z - 3 * left));
  }
  static __device__ __forceinline__ uint32_t bytes(uint32_t v) { return __builtin_amdgcn_perm(v, v, 0u); }
  static __device__ __forceinline__ float times(uint32_t v) { return fmaf((float)(v >> 8 & 255u), 0x1p-6f, 1.0f); }
};

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
// part: of int4_gemm_workspace bytes.
hipError_t launch_int4_gemm(const Int4Gemm& a, float* part, hipStream_t s);
size_t int4_gemm_workspace(int64_t m, int64_t n, int64_t k);

// The experts' products, rows being places: h[place, f] = silu(x Wg^T) (x Wu^T) of the pair's token, in
// bf16; part[pair, d] = h[place] Wd^T, in fp32.  bf16 is what the matrix instructions of the down product take beside
// bf16 weights, and h is rounded so for every number of tokens: the block's error is 2.4e-3 of its output's size, where
// h in fp32 would leave 1.7e-3, the output's own rounding.
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
// Few tokens: a pair at a time (launch_int4_vec_experts), each streaming its expert's weights, unless there are so many
// more pairs than experts that at least 25 MB of them are read again whatever the ids, which takes as long as ordering
// the pairs and joining their outputs.  The ids are on the GPU, so how many pairs share an expert is not known here.
// 64 experts of 4096 x 1792 (11 MB each), a pair at a time and ordered, us: 16 pairs 41 and 55, 32 71 and 89, 64 133
// and 133 (all alike: 42 experts, 245 MB read again, from caches); 64 that are all for one expert 113 and 38.
bool int4_experts_by_pairs(int64_t tokens, int64_t pairs, int64_t experts, int64_t d, int64_t f);

// The kernels.  sp24_int4_vec.hip: one or two tokens; the experts' block with pairs in their own order, y being
// its output.
hipError_t launch_int4_vec(const Int4Gemm& g, hipStream_t s);
hipError_t launch_int4_vec_experts(const Int4Experts& e, const int32_t* ids, const float* weights, uint16_t* y,
                                   hipStream_t s);
constexpr int kSlabTokens = 1024;  // dense products: beyond, the tiled kernel is always the faster
// sp24_int4_slab.hip: 16 mb tokens a workgroup, its waves along the columns (32 each; GATED: 16) and along K, the
// values of K of a workgroup (k or more: no slices) and of a pass; multiples of 128.
struct SlabPlan {
  int mb, cbs, kp, slice, chunk;
};
// part: fp32 [slices, m, n], with slices
hipError_t launch_int4_slab(const SlabPlan& q, const Int4Gemm& g, float* part, hipStream_t s);
hipError_t launch_int4_slab_gated(const SlabPlan& q, const Int4Experts& e, hipStream_t s);
hipError_t launch_int4_slab_down(const SlabPlan& q, const Int4Experts& e, hipStream_t s);
// sp24_int4_tiled.hip: tiles of 256 x 256 (cfg 0) or 128 x 128 (cfg 1).
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

// Tiles of up to BM places by columns: `number` counts, expert after expert, column tile after column tile and
// in each all of the expert's row tiles (which read the same rows of W).  False past the last.  Every lane of
// the wave gets the same answer.
template <int BM>
__device__ __forceinline__ bool find_tile(const Pairs& p, int number, int columns, int lane, int& expert, int& first,
                                          int& rows, int& column) {
  int base = 0;
  for (int c = 0; c < p.experts; c += 64) {
    const int e = c + lane;
    const int lo = e < p.experts ? p.offsets[e] : 0, hi = e < p.experts ? p.offsets[e + 1] : 0;
    int upto = (hi - lo + BM - 1) / BM * columns;  // of experts c .. e
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    const uint64_t past = __ballot(number < base + upto);
    if (past != 0) {
      const int at = __ffsll((unsigned long long)past) - 1;
      const int start = at == 0 ? base : base + __shfl(upto, at - 1);
      const int begin = __shfl(lo, at), end = __shfl(hi, at), tiles = (end - begin + BM - 1) / BM;
      expert = c + at;
      column = (number - start) / tiles;
      first = begin + (number - start - column * tiles) * BM;
      rows = min(BM, end - first);
      return true;
    }
    base += __shfl(upto, 63);
  }
  return false;
}

// The number of such tiles.  Every lane of the wave gets the same answer.
template <int BM>
__device__ __forceinline__ int count_tiles(const Pairs& p, int lane) {
  int tiles = 0;
  for (int e = lane; e < p.experts; e += 64) tiles += (p.offsets[e + 1] - p.offsets[e] + BM - 1) / BM;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) tiles += __shfl_xor(tiles, o);
  return tiles;
}

// A bound of the number of such tiles that needs no look at the ids.
inline int64_t most_tiles(int64_t pairs, int experts, int bm) {
  const int64_t used = pairs < experts ? pairs : experts;  // each has one that is not full
  return (pairs - used) / bm + used;
}

}  // namespace sp24
