// Products with integer 4-bit weights for one or two tokens, and the experts' block for a few, pair by
// pair: the weight's bytes are the time.
//
// A workgroup holds 8 rows of W, a wave of it a chunk of 2048 values of K, lane l of it the 32 values of block l: each
// row's load is 1 KB of neighbouring bytes, and the lane's x stays in registers for all rows.  No LDS
// before the end, no waits between waves: what is in flight at once is a decode step's whole share of
// W (n = 14336, k = 4096: 14 waves a CU of 8 KB each).
// Two values at a time: c + q - z as bf16 pairs (shift, and-or; with zero points their bytes), then
// v_dot2_f32_bf16, 11 instructions for 8 values and one token, or 13.  The sum of c x and the group's scale come in
// behind the block's sum, in fp32; a block of 32 lies in one group.
// The lanes' sums are joined by register exchanges (rows and lanes transposed on the way), those of
// the chunks through LDS, in a fixed order; the experts' down product keeps the slots of a token apart until each
// is finished, then adds them in their order, times their weights.
//
// One token of 14336 x 4096 (30.3 MB) takes 6.8 to 7.1 us (4.3 to 4.5 TB/s; a copy reaches 5.2), a call after
// another 7.1; two tokens 8.9 in a graph, as many again of the products.  The experts' block of one
// token, 8 of 64 experts of 4096 x 1792: gated 11.8 to 12.2 us (60 MB: 5 TB/s), down 8.2 to 8.4.  8 rows a
// workgroup: with 4 each lane's x would be read twice as often; 16 leave fewer waves than fill the CUs.
#include "sp24_int4.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

enum { PLAIN = 0, GATED = 1, DOWN = 2 };

struct Args {
  int n, k, group;  // n: output columns (GATED: W has 2 n rows an expert)
  const uint16_t* x;
  Int4Weight w;
  uint16_t* y;
  // GATED, DOWN: pairs in their own order (pair t * top + j)
  const int32_t* ids;
  const float* weights;
  int experts, top;
  int kw;              // waves of a workgroup, along K
};

// Two values of all lanes into one: a's sum over lanes OFF apart where lane & OFF is 0, b's where not.
template <int OFF>
__device__ __forceinline__ float merge(float a, float b, int lane) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  if constexpr (OFF == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(ua, ub, false, false);
    return __uint_as_float((uint32_t)r[0]) + __uint_as_float((uint32_t)r[1]);
  } else if constexpr (OFF == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(ua, ub, false, false);
    return __uint_as_float((uint32_t)r[0]) + __uint_as_float((uint32_t)r[1]);
  } else {  // 8: a row of 16 lanes rotated by 8
    const float keep = lane & 8 ? b : a, send = lane & 8 ? a : b;
    return keep + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(send), 0x128, 0xF, 0xF,
                                                                       true));
  }
}

__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
}

constexpr int RB = 8;  // rows of W a workgroup (GATED: half of them gate rows, half their up rows)

// MT tokens.
template <int MT, int MODE, int OCC, bool Z>
__global__ __launch_bounds__(512, OCC) void int4_vec_kernel(Args p) {
  constexpr int OUT = MODE == GATED ? RB / 2 : RB;  // outputs a workgroup
  static_assert(MODE == PLAIN || MT == 1, "a pair has one token");
  constexpr int TOP = 64;  // the most slots of a token that sp24_experts_int4 takes
  __shared__ float red[MODE == DOWN ? TOP * 8 : 8][RB * MT];  // by wave; DOWN: by slot and wave
  __shared__ float slot_weight[MODE == DOWN ? TOP : 1];
  __shared__ int slot_there[MODE == DOWN ? TOP : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int kw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nblocks = (p.n + OUT - 1) / OUT;
  const int64_t item = blockIdx.x / nblocks;  // PLAIN: 0; GATED: a pair; DOWN: a token
  const int n0 = (int)(blockIdx.x % nblocks) * OUT;
  const int blocks = p.k / 32, chunks = (blocks + 63) / 64, groups = p.k / p.group;
  const int gshift = p.group == 32 ? 0 : p.group == 64 ? 1 : 2;
  const size_t half = (size_t)p.k / 2;
  size_t expert = 0;
  if constexpr (MODE == GATED) {
    const int id = p.ids[item];
    if ((uint32_t)id >= (uint32_t)p.experts) return;
    expert = id;
  }

  int slot_id = 0;  // DOWN: of slot `tid`, loaded here and looked at behind the products
  float weight = 0.0f;
  if constexpr (MODE == DOWN) {
    if (tid < p.top) {
      slot_id = p.ids[item * p.top + tid];
      weight = p.weights[item * p.top + tid];
    }
  }

  const Int4Bits<Z> bits;
  float acc[RB][MT];
  auto clear = [&] {
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[r][t] = 0.0f;
  };
  // The lanes' sums, to red[at]: rows 2^0, 2^1, 2^2 go to lane bits 5, 4, 3.
  auto join = [&](int at) {
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      float v[RB / 2];
#pragma unroll
      for (int r = 0; r < RB / 2; ++r) v[r] = merge<32>(acc[2 * r][t], acc[2 * r + 1][t], lane);
      const float u = merge<8>(merge<16>(v[0], v[1], lane), merge<16>(v[2], v[3], lane), lane);
      const int row = (lane >> 5 & 1) | (lane >> 4 & 1) << 1 | (lane >> 3 & 1) << 2;
      const uint32_t f =
          fold_lanes<4>(fold_lanes<2>(fold_lanes<1>(__float_as_uint(u), bits_sum), bits_sum), bits_sum);
      if ((lane & (64 / RB - 1)) == 0) red[at][row * MT + t] = __uint_as_float(f);
    }
  };
  clear();

  // DOWN: chunk after chunk of slot after slot, the waves in turn
  const int work = MODE == DOWN ? chunks * p.top : chunks;
  for (int c = kw; c < work; c += p.kw) {
    int chunk = c, slot = 0;
    const uint16_t* xr = p.x;
    if constexpr (MODE == DOWN) {
      slot = c / chunks;
      chunk = c - slot * chunks;
      const int id = p.ids[item * p.top + slot];
      if ((uint32_t)id >= (uint32_t)p.experts) continue;  // uniform
      expert = id;
      xr += (size_t)(item * p.top + slot) * p.k;
    } else if constexpr (MODE == GATED) {
      xr += (size_t)(item / p.top) * p.k;
    }
    const int b = chunk * 64 + lane, kb = min(b, blocks - 1);

    // All loads before the first product; X's first, since loads arrive in order and a row of W is multiplied while
    // the rows behind it are on their way.
    u32x4 x[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const size_t tok = MODE == PLAIN ? t : 0;
      const u32x4* xp = reinterpret_cast<const u32x4*>(xr + tok * p.k + (size_t)kb * 32);
#pragma unroll
      for (int d = 0; d < 4; ++d) x[t][d] = xp[d];
    }
    u32x4 w[RB];
    uint32_t s[RB], z[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int col = min(n0 + (MODE == GATED ? r % OUT : r), p.n - 1) + (MODE == GATED && r >= OUT ? p.n : 0);
      const size_t row = expert * (MODE == GATED ? 2 * (size_t)p.n : (size_t)p.n) + col;
      w[r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p.w.codes + row * half) + kb);
      const size_t g = row * groups + (kb >> gshift);
      s[r] = p.w.scales[g];
      z[r] = Z ? p.w.zeros[g] : 0;
    }
    __builtin_amdgcn_sched_barrier(0);
    float cx[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      cx[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[t][d][i] = b < blocks ? x[t][d][i] : 0u;  // past the row: nothing is added
          cx[t] = dot2(Int4Bits<Z>::kConstant, x[t][d][i], cx[t]);
        }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const uint32_t zero = Z ? Int4Zeros::of(z[r]) : 0, zp = Z ? Int4Zeros::bytes(zero) : 0;
      float sum[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) sum[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const u32x4 q = __builtin_bit_cast(u32x4, bits.values(w[r][d], zp));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int t = 0; t < MT; ++t) sum[t] = dot2(q[i], x[t][d][i], sum[t]);
      }
      const float scale = bf16_to_f32(s[r]), times = Z ? Int4Zeros::times(zero) : 1.0f;
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[r][t] += scale * (Z ? sum[t] - times * cx[t] : sum[t] - cx[t]);
    }
    if constexpr (MODE == DOWN) {
      if (c + p.kw >= (slot + 1) * chunks) {  // the last of the slot's that this wave has
        join(slot * 8 + kw);
        clear();
      }
    }
  }

  if constexpr (MODE == DOWN) {
    if (tid < TOP) {
      slot_weight[tid] = weight;
      slot_there[tid] = tid < p.top && (uint32_t)slot_id < (uint32_t)p.experts;
    }
    __syncthreads();
    // the slots in their order: each one's product, its chunks in their order, times its weight
    if (tid < RB) {
      constexpr int J = 8;  // slots whose values are read together, without branches between
      const int parts = min(chunks, p.kw);
      float y = 0.0f;
#pragma unroll 1
      for (int j0 = 0; j0 < p.top; j0 += J) {
        float v[J], w[J];
        int there[J];
#pragma unroll
        for (int i = 0; i < J; ++i) {
          w[i] = slot_weight[j0 + i];
          there[i] = slot_there[j0 + i];
          v[i] = red[(j0 + i) * 8 + ((j0 + i) * chunks & 7)][tid];
        }
#pragma unroll 1
        for (int part = 1; part < parts; ++part)
#pragma unroll
          for (int i = 0; i < J; ++i)
            v[i] += red[(j0 + i) * 8 + (((j0 + i) * chunks + part) & 7)][tid];  // fewer than 8 waves: a chunk each
#pragma unroll
        for (int i = 0; i < J; ++i) y += (there[i] != 0 ? w[i] : 0.0f) * (there[i] != 0 ? v[i] : 0.0f);
      }
      if (n0 + tid < p.n) p.y[(size_t)item * p.n + n0 + tid] = (uint16_t)f32x2_to_bf16x2(y, 0.0f);
    }
    return;
  }
  join(kw);
  __syncthreads();
  if (tid < OUT * MT) {
    const int t = tid % MT, i = tid / MT;
    float v = 0.0f, u = 0.0f;
    for (int z = 0; z < p.kw; ++z) {
      v += red[z][i * MT + t];
      if constexpr (MODE == GATED) u += red[z][(i + OUT) * MT + t];
    }
    if constexpr (MODE == GATED) v = silu_mul(v, u);
    const int64_t row = MODE == PLAIN ? t : item;  // GATED: the pair
    if (n0 + i < p.n)
      p.y[(size_t)row * p.n + n0 + i] = (uint16_t)f32x2_to_bf16x2(v, 0.0f);
  }
}

template <int MT, int MODE, int OCC>
hipError_t launch(Args a, int64_t items, hipStream_t s) {
  constexpr int OUT = MODE == GATED ? RB / 2 : RB;
  const int work = (a.k / 32 + 63) / 64 * (MODE == DOWN ? a.top : 1);
  a.kw = work < 8 ? work : 8;
  const int64_t grid = items * ((a.n + OUT - 1) / OUT);
  if (grid * 64 * a.kw >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;  // HIP counts threads in 32 bits
  const dim3 g((uint32_t)grid), block(64 * a.kw);
  if (a.w.zeros != nullptr) hipLaunchKernelGGL((int4_vec_kernel<MT, MODE, OCC, true>), g, block, 0, s, a);
  else hipLaunchKernelGGL((int4_vec_kernel<MT, MODE, OCC, false>), g, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int4_vec(const Int4Gemm& g, hipStream_t s) {
  const Args a{g.n, g.k, g.group, g.x, g.w, g.y, nullptr, nullptr, 1, 1, 0};
  return g.m == 1 ? launch<1, PLAIN, 5>(a, 1, s) : launch<2, PLAIN, 4>(a, 1, s);
}

hipError_t launch_int4_vec_experts(const Int4Experts& e, const int32_t* ids, const float* weights, uint16_t* y,
                                   hipStream_t s) {
  const Args gated{e.f, e.d, e.group, e.x, e.gu, e.h, ids, weights, e.pairs.experts, e.pairs.top, 0};
  const hipError_t st = launch<1, GATED, 5>(gated, e.pairs.count, s);
  if (st != hipSuccess) return st;
  const Args down{e.d, e.f, e.group, e.h, e.down, y, ids, weights, e.pairs.experts, e.pairs.top, 0};
  return launch<1, DOWN, 4>(down, e.tokens, s);
}

}  // namespace sp24
