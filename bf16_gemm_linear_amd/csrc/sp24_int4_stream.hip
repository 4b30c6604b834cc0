// Products with integer 4-bit weights for up to 64 tokens (or an expert's few): the weight's bytes are
// the time.
//
// A workgroup owns up to 16 RBK rows of W (GATED: half of them gate rows, half their up rows), up to
// 16 MB rows of X and all of K.  Its 8 waves take turns at pieces of 256 values and wait for nobody until the end;
// each loads its operands straight into registers, one step of 128 values (U of them) ahead of the one it
// multiplies.  The waves' sums are joined through LDS in a fixed order.
//
// v_mfma_f32_16x16x32_bf16, A = X, B = W: lane l holds row l % 16 and values 8 (l / 16) .. + 7 of a block of
// 32; accumulator register e is token 4 (l / 16) + e, W row l % 16.  A lane loads 16 bytes of codes, block
// l / 16 of its row's four; a transposition of the 4 x 4 words of lanes l, l + 16, l + 32, l + 48 (four
// register exchanges) gives it word l / 16 of every block, so each instruction covers one block of 32 and
// any group size works.  Codes become the bf16 pairs (128 + q); what that adds, 128 + z times the sum of
// x, is taken off in fp32 behind a group's sum, the sum of x coming from one more instruction
// with ones.  Rows past the last are the last one again; their outputs are not stored.
#include "sp24_int4.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

enum { PLAIN = 0, GATED = 1, DOWN = 2 };

struct Args {
  int m, n, k, group;
  const uint16_t* x;
  Int4Weight w;
  uint16_t* y;
  float* part;
  Pairs pairs;
  int cols;  // output columns a workgroup (at most 16 RBK, GATED 8 RBK)
};

// registers i of lanes l, l + 16, l + 32, l + 48: element (i, lane group) goes to (lane group, i)
__device__ __forceinline__ void transpose4(uint32_t (&v)[4]) {
  auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap((uint32_t)a[0], (uint32_t)b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap((uint32_t)a[1], (uint32_t)b[1], false, false);
  v[0] = c[0];
  v[1] = c[1];
  v[2] = d[0];
  v[3] = d[1];
}

template <int RBK, int MB>
struct Step {
  u32x4 w[RBK], x[MB][4];
};

constexpr int kScaleWords = 8192;  // scales of a workgroup that are in LDS at a time
constexpr int F = 8;               // of them, those that a thread loads at a time

// G128: a scale covers a whole step; otherwise it is applied every 32 values.  S: steps in flight.
template <int RBK, int MB, int KW, int S, int MODE, bool G128, int OCC>
__global__ __launch_bounds__(KW * 64, OCC) void int4_stream_kernel(Args p) {
  constexpr int OB = MODE == GATED ? RBK / 2 : RBK;  // row blocks of the output
  constexpr int H = MODE == GATED ? 2 : 1;           // gate rows, up rows
  static_assert(OB > 0, "GATED needs a gate and an up block");
  constexpr int RED = KW * RBK * MB * 1024, SCALES = (kScaleWords + 16 * RBK) * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[RED > SCALES ? RED : SCALES];
  uint32_t* const sz = reinterpret_cast<uint32_t*>(lds);  // scale and zero of (row, group): bf16, byte
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int kw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nblocks = (p.n + p.cols - 1) / p.cols;
  const int n0 = (int)(blockIdx.x % nblocks) * p.cols, tile = (int)(blockIdx.x / nblocks);
  const int ncols = min(p.cols, p.n - n0);
  int expert = 0, first = tile * 16 * MB, rows = min(16 * MB, p.m - first);
  if constexpr (MODE != PLAIN)
    if (!find_tile<16 * MB>(p.pairs, tile, lane, expert, first, rows)) return;

  // Per-lane offsets are 32-bit from uniform bases (k <= 2^20, at most 64 rows).
  const int half = p.k / 2, groups = p.k / p.group, blocks = p.k / 32;
  const int gshift = p.group == 32 ? 0 : p.group == 64 ? 1 : 2;
  const size_t row0 = (size_t)expert * (H * p.n) + n0;
  const uint8_t *codes[H], *zeros[H];
  const uint16_t* scales[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const size_t row = row0 + (size_t)h * p.n;
    codes[h] = p.w.codes + row * half;
    scales[h] = p.w.scales + row * groups;
    zeros[h] = p.w.zeros == nullptr ? nullptr : p.w.zeros + row * groups;
  }
  uint32_t wrow[OB];
#pragma unroll
  for (int i = 0; i < OB; ++i) wrow[i] = (uint32_t)min(16 * i + r, ncols - 1) * (uint32_t)half;
  // X: PLAIN and DOWN 32-bit offsets from the tile's first row, GATED any rows
  const uint16_t* const x0 = p.x + (size_t)(MODE == GATED ? 0 : first) * p.k;
  size_t xoff[MB];
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    const int row = min(16 * j + r, rows - 1);
    if constexpr (MODE == GATED) xoff[j] = (size_t)(p.pairs.order[first + row] / p.pairs.top) * p.k + 8 * q;
    else xoff[j] = (uint32_t)(row * p.k + 8 * q);
  }

  f32x4 acc[RBK][MB];
#pragma unroll
  for (int i = 0; i < RBK; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const f32x4 zero{0.f, 0.f, 0.f, 0.f};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

  // K in chunks whose scales fit: whole steps, since kScaleWords / (16 RBK) groups are a multiple of 256 values
  constexpr int GC = kScaleWords / (16 * RBK);
  for (int g0 = 0; g0 < groups; g0 += GC) {
    const int gc = min(GC, groups - g0), stride = gc | 1;  // odd: the rows' words lie in different banks
    const int first_block = g0 << gshift, last = min(blocks, (g0 + gc) << gshift);  // blocks of 32 of this chunk
    const int steps = (last - first_block + 3) / 4;
    // this wave's step t of the chunk: pieces of two steps, the waves in turn
    auto number = [&](int t) { return (t / 2 * KW + kw) * 2 + t % 2; };
    auto load = [&](Step<RBK, MB>& s, int t) {
      const int b0 = first_block + 4 * min(number(t), steps - 1);
      const uint32_t at = 16u * (uint32_t)min(b0 + q, blocks - 1);  // this lane's block of its row's four
#pragma unroll
      for (int i = 0; i < RBK; ++i)
        s.w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes[i / OB] + (wrow[i % OB] + at)));
#pragma unroll
      for (int j = 0; j < MB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint16_t* const xb = x0 + 32 * min(b0 + i, blocks - 1);
          if constexpr (MODE == GATED) s.x[j][i] = *reinterpret_cast<const u32x4*>(xb + xoff[j]);
          else s.x[j][i] = *reinterpret_cast<const u32x4*>(xb + (uint32_t)xoff[j]);
        }
    };
    auto compute = [&](Step<RBK, MB>& s, int t) {
      const int b0 = first_block + 4 * number(t), left = last - b0;  // uniform; blocks of this step
      if (left <= 0) return;
      const uint32_t* const szr = sz + r * stride + ((b0 >> gshift) - g0);
      if constexpr (G128) {  // then left >= 4
        f32x4 sx[MB];
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          sx[j] = zero;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sx[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, s.x[j][i]), ones, sx[j], 0, 0, 0);
        }
#pragma unroll
        for (int rb = 0; rb < RBK; ++rb) {
          const uint32_t both = szr[16 * rb * stride];
          uint32_t w[4] = {s.w[rb][0], s.w[rb][1], s.w[rb][2], s.w[rb][3]};
          transpose4(w);
          f32x4 v[MB];
#pragma unroll
          for (int j = 0; j < MB; ++j) v[j] = zero;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bf16x8 b = __builtin_bit_cast(
                bf16x8, u32x4{int4_pair(w[i], 0), int4_pair(w[i], 1), int4_pair(w[i], 2), int4_pair(w[i], 3)});
#pragma unroll
            for (int j = 0; j < MB; ++j)
              v[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, s.x[j][i]), b, v[j], 0, 0, 0);
          }
          const float sc = __uint_as_float(both & 0xFFFF0000u), zp = 128.0f + (float)(both & 255u);
#pragma unroll
          for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[rb][j][e] += sc * (v[j][e] - zp * sx[j][e]);
        }
      } else {
        uint32_t w[RBK][4];
#pragma unroll
        for (int rb = 0; rb < RBK; ++rb) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[rb][i] = s.w[rb][i];
          transpose4(w[rb]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i >= left) break;  // uniform
          f32x4 sx[MB];
#pragma unroll
          for (int j = 0; j < MB; ++j)
            sx[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, s.x[j][i]), ones, zero, 0, 0, 0);
#pragma unroll
          for (int rb = 0; rb < RBK; ++rb) {
            const uint32_t both = szr[16 * rb * stride + (i >> gshift)];
            const bf16x8 b = __builtin_bit_cast(bf16x8, u32x4{int4_pair(w[rb][i], 0), int4_pair(w[rb][i], 1),
                                                              int4_pair(w[rb][i], 2), int4_pair(w[rb][i], 3)});
            const float sc = __uint_as_float(both & 0xFFFF0000u), zp = 128.0f + (float)(both & 255u);
#pragma unroll
            for (int j = 0; j < MB; ++j) {
              const f32x4 v =
                  __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, s.x[j][i]), b, zero, 0, 0, 0);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[rb][j][e] += sc * (v[e] - zp * sx[j][e]);
            }
          }
        }
      }
    };

    // The scales: up to 64 lanes along the groups, the rest of the threads along the rows, F rows a
    // thread at a time.  The last loads go out before the first steps', and into LDS behind them.
    int ashift = 6;
    while (ashift > 0 && (1 << ashift) / 2 >= gc) --ashift;
    const int fg = tid & ((1 << ashift) - 1), frow = tid >> ashift, per = (KW * 64) >> ashift;
    uint32_t fs[F], fz[F];
    auto fetch = [&](int row0, int g) {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int row = min(row0 + f * per, 16 * RBK - 1), h = row / (16 * OB);
        const uint32_t at =
            (uint32_t)min(row - 16 * OB * h, ncols - 1) * (uint32_t)groups + (uint32_t)(g0 + min(g, gc - 1));
        fs[f] = (H == 2 && h == 1 ? scales[H - 1] : scales[0])[at];
        fz[f] = p.w.zeros == nullptr ? kInt4Zero : (H == 2 && h == 1 ? zeros[H - 1] : zeros[0])[at];
      }
    };
    auto store = [&](int row0, int g) {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int row = row0 + f * per;
        if (row < 16 * RBK && g < gc) sz[row * stride + g] = fs[f] << 16 | fz[f];
      }
    };
    if (g0 > 0) __syncthreads();  // the chunk before is done with its scales
    int fr = frow, g = fg;
    for (;;) {
      fetch(fr, g);
      if (fr - frow + F * per >= 16 * RBK && g - fg + (1 << ashift) >= gc) break;  // uniform
      store(fr, g);
      fr += F * per;
      if (fr - frow >= 16 * RBK) {
        fr = frow;
        g += 1 << ashift;
      }
    }
    __builtin_amdgcn_sched_barrier(0);

    const int pieces = (steps + 1) / 2;
    const int mine = pieces > kw ? (pieces - kw + KW - 1) / KW * 2 : 0;  // steps, at most one of them past the end
    Step<RBK, MB> st[S];
    if (mine > 0) {
#pragma unroll
      for (int u = 0; u < S; ++u) load(st[u], u);
    }
    __builtin_amdgcn_sched_barrier(0);
    store(fr, g);
    __syncthreads();
    int t = 0;
    for (; t + 2 * S <= mine; t += S) {
#pragma unroll
      for (int u = 0; u < S; ++u) {
        compute(st[u], t + u);
        __builtin_amdgcn_sched_barrier(0);
        load(st[u], t + u + S);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (t < mine) {
#pragma unroll
      for (int u = 0; u < S; ++u) {
        if (t + u < mine) compute(st[u], t + u);
        if (t + u + S < mine) load(st[u], t + u + S);
      }
#pragma unroll
      for (int u = 0; u < S; ++u)
        if (t + u + S < mine) compute(st[u], t + u + S);
    }
  }

  __syncthreads();
  f32x4(*red)[RBK * MB][64] = reinterpret_cast<f32x4(*)[RBK * MB][64]>(lds);
#pragma unroll
  for (int i = 0; i < RBK; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) red[kw][i * MB + j][lane] = acc[i][j];
  __syncthreads();
  auto sum = [&](int at, int l) {
    f32x4 v = red[0][at][l];
#pragma unroll
    for (int z = 1; z < KW; ++z) v += red[z][at][l];
    return v;
  };
  for (int t = tid; t < OB * MB * 64; t += KW * 64) {
    const int l = t & 63, j = t / 64 % MB, i = t / 64 / MB;
    f32x4 v = sum(i * MB + j, l);
    if constexpr (MODE == GATED) {
      const f32x4 u = sum((i + OB) * MB + j, l);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = silu_mul(v[e], u[e]);
    }
    const int col = 16 * i + (l & 15);
    if (col >= ncols) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 16 * j + 4 * (l >> 4) + e;
      if (row >= rows) continue;
      if constexpr (MODE == DOWN) p.part[(size_t)p.pairs.order[first + row] * p.n + n0 + col] = v[e];
      else p.y[(size_t)(first + row) * p.n + n0 + col] = (uint16_t)f32x2_to_bf16x2(v[e], 0.0f);
    }
  }
}

template <int RBK, int MB, int KW, int S, int OCC, int MODE>
hipError_t launch(Args a, int64_t tiles, hipStream_t s) {
  const int64_t grid = tiles * ((a.n + a.cols - 1) / a.cols);
  if (grid * KW * 64 >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;  // HIP counts threads in 32 bits
  if (a.group == 128)
    hipLaunchKernelGGL((int4_stream_kernel<RBK, MB, KW, S, MODE, true, OCC>), dim3((uint32_t)grid), dim3(KW * 64), 0, s,
                       a);
  else
    hipLaunchKernelGGL((int4_stream_kernel<RBK, MB, KW, S, MODE, false, OCC>), dim3((uint32_t)grid), dim3(KW * 64), 0,
                       s, a);
  return hipGetLastError();
}

// rb: row blocks of 16 a workgroup; mb: tokens / 16 a workgroup
template <int MODE>
hipError_t by_size(int rb, int mb, const Args& a, int64_t tiles, hipStream_t s) {
  switch (10 * rb + mb) {
    case 11: if constexpr (MODE != GATED) return launch<1, 1, 4, 6, 2, MODE>(a, tiles, s); break;
    case 12: if constexpr (MODE != GATED) return launch<1, 2, 4, 4, 2, MODE>(a, tiles, s); break;
    case 14: if constexpr (MODE != GATED) return launch<1, 4, 4, 2, 2, MODE>(a, tiles, s); break;
    case 21: return launch<2, 1, 4, 5, 2, MODE>(a, tiles, s);
    case 22: return launch<2, 2, 4, 3, 2, MODE>(a, tiles, s);
    case 24: return launch<2, 4, 4, 2, 2, MODE>(a, tiles, s);
    case 41: return launch<4, 1, 4, 4, 2, MODE>(a, tiles, s);
    case 42: return launch<4, 2, 4, 3, 2, MODE>(a, tiles, s);
  }
  return hipErrorInvalidConfiguration;
}

}  // namespace

hipError_t launch_int4_stream(int rb, int mb, int cols, const Int4Gemm& g, hipStream_t s) {
  const Args a{g.m, g.n, g.k, g.group, g.x, g.w, g.y, nullptr, Pairs{}, cols};
  return by_size<PLAIN>(rb, mb, a, (g.m + 16 * mb - 1) / (16 * mb), s);
}

hipError_t launch_int4_stream_gated(int rb, int mb, int cols, const Int4Experts& e, hipStream_t s) {
  const Args a{0, e.f, e.d, e.group, e.x, e.gu, e.h, nullptr, e.pairs, cols};
  return by_size<GATED>(rb, mb, a, most_tiles(e.pairs.count, e.pairs.experts, 16 * mb), s);
}

hipError_t launch_int4_stream_down(int rb, int mb, int cols, const Int4Experts& e, hipStream_t s) {
  const Args a{0, e.d, e.f, e.group, e.h, e.down, nullptr, e.part, e.pairs, cols};
  return by_size<DOWN>(rb, mb, a, most_tiles(e.pairs.count, e.pairs.experts, 16 * mb), s);
}

}  // namespace sp24
