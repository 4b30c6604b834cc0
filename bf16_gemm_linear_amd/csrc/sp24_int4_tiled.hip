// Products with integer 4-bit weights for many tokens, over LDS tiles: the matrix instructions are the
// time.
//
// A workgroup owns BM rows of X by BN rows of W (GATED: per wave 32 gate rows and their up rows) and
// walks K in steps of 64 values with two buffers in LDS: X straight from global memory (global_load_lds), W
// through registers, where a thread widens 32 codes of a row to bf16 for the next step while
// this one is multiplied: every code is widened once for BM rows of X.
//
// No value of W is rounded: with a group's scale as m 2^e, 1 <= m < 2, what is multiplied is (q - z) 2^e, which
// bf16 holds exactly, and the sums are kept in units of the group's m: where a group ends they are multiplied by
// m / m', between 1/2 and 2, one instruction a sum and group, and by the last m at the end.  (A second
// set of accumulators for a group's sums does not fit beside the 256 x 256 tile's first; rounding
// (q - z) s to bf16 instead takes less time, but its errors, 2^-9 of each, were up to 3 half steps of bf16
// where a few channels of X are 20 times as large as the others.)
//
// v_mfma_f32_32x32x16_bf16, A = X, B = W: lane l holds row l % 32 and values 8 (l / 32) .. + 7;
// accumulator register 4 g + e is token 8 g + 4 (l / 32) + e, W row l % 32.  LDS rows of 128 bytes are
// XOR-swizzled in pieces of 16; the swizzle of X is applied on the global side.
//
// 2047 x 28672 x 8192 takes 0.98 to 1.08 ms (890 to 980 TFLOP/s; the library's bf16 product of that size, without
// anything to widen and with four times the bytes of W, 0.68 to 0.78), its matrix cores busy 42% of the cycles: with 64 KB a step and all registers taken there is
// one workgroup a CU, whose waves meet at every step.  Tiles of 128 x 128, two workgroups a CU, widen every code
// twice as often; they win where 256 x 256 would leave CUs idle (the table beside the experts' plan).
#include <type_traits>

#include "sp24_dma.hpp"
#include "sp24_int4.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

enum { PLAIN = 0, GATED = 1, DOWN = 2 };
constexpr int KS = 64, RB = KS * 2, P = RB / 16;  // a step: values, bytes and 16-byte pieces of a row

struct Args {
  int m, n, k, group;
  const uint16_t* x;
  Int4Weight w;
  uint16_t* y;
  float* part;
  Pairs pairs;
  int tiles, nblocks;  // row tiles (at most) and column tiles
};

// Two buffers of X and of W in LDS; W's codes are in registers two steps ahead.
template <int BM_, int BN_, int WM_, int WN_>
struct TileCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int NT = WM * WN * 64, TI = BM / WM / 32, TJ = BN / WN / 32;
  static constexpr int X_I = BM / 8 / (WM * WN);  // load instructions of X a wave and step
  static constexpr int X_BYTES = BM * RB, W_BYTES = BN * RB, W_OFF = 2 * X_BYTES, M_OFF = W_OFF + 2 * W_BYTES;
  static constexpr int ROW_OFF = M_OFF + 2 * 2 * BN * 4;  // behind m of every row's two blocks of 32, two buffers
  static constexpr int LDS = ROW_OFF + BM * 4;            // and the pair of every row
  static_assert(X_I * 8 * WM * WN == BM && NT == BN * 2 && TI > 0 && TJ > 0 && LDS <= 160 * 1024, "tile");
};

// 8 codes -> 8 bf16 values (q - z) s; ns = -z s, s a power of two.
__device__ __forceinline__ u32x4 widen(uint32_t w, float s, float ns) {
  uint32_t e = w & 0x0F0F0F0Fu, o = (w >> 4) & 0x0F0F0F0Fu;
  asm("" : "+v"(e), "+v"(o));  // or the compiler takes the codes out of w one by one: an instruction more for most
  // bytes of e: values 0 4 1 5, of o: 2 6 3 7
  auto f = [&](uint32_t b, int i) { return fmaf((float)((b >> (8 * i)) & 255u), s, ns); };
  return u32x4{f32x2_to_bf16x2(f(e, 0), f(e, 2)), f32x2_to_bf16x2(f(o, 0), f(o, 2)),
               f32x2_to_bf16x2(f(e, 1), f(e, 3)), f32x2_to_bf16x2(f(o, 1), f(o, 3))};
}

template <class C, int MODE, int G>
__global__ __launch_bounds__(C::NT, 2) void int4_tiled_kernel(Args p) {
  constexpr int TI = C::TI, TJ = C::TJ, H = MODE == GATED ? 2 : 1;
  static_assert(MODE != GATED || TJ == 2, "a wave's gate tile and its up tile");
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;

  // Workgroups go to the 8 XCDs in turn; each XCD takes a run of tiles, all row tiles of a column
  // tile next to each other, so that its L2 holds the W and X that they share.
  int tiles = p.tiles;
  if constexpr (MODE != PLAIN) tiles = count_tiles<C::BM>(p.pairs, lane);  // the grid is for the most there can be
  const int total = tiles * p.nblocks, run = (total + 7) / 8;
  const int number = (int)(blockIdx.x % 8) * run + (int)(blockIdx.x / 8);
  if ((int)(blockIdx.x / 8) >= run || number >= total) return;
  int expert = 0, first, rows, nb;
  if constexpr (MODE == PLAIN) {
    first = number % p.tiles * C::BM;
    nb = number / p.tiles;
    rows = min(C::BM, p.m - first);
  } else {
    if (!find_tile<C::BM>(p.pairs, number, p.nblocks, lane, expert, first, rows, nb)) return;
  }
  const int n0 = nb * (C::BN / H);

  int* const pair_of = reinterpret_cast<int*>(lds + C::ROW_OFF);  // DOWN: the pair of every row
  if constexpr (MODE == DOWN)
    for (int i = tid; i < rows; i += C::NT) pair_of[i] = p.pairs.order[first + i];

  const int steps = (p.k + KS - 1) / KS;
  // Loads past the last step are that step's again, so that every step has the same number of them.  A last
  // step of 32 values (groups of 32 alone) has its first half twice: the second meets values of W that are 0.
  auto begin = [&](int t) { return min(t, steps - 1) * KS; };
  auto half_step = [&](int k0) { return G == 32 && k0 + KS > p.k; };  // uniform
  // X: this lane's rows (of 8 an instruction) and swizzled pieces, from uniform bases: PLAIN and DOWN 32-bit
  // offsets (k <= 2^20, at most 256 rows)
  const uint16_t* const x0 = MODE == GATED ? p.x : p.x + (size_t)first * p.k;
  using Offset = std::conditional_t<MODE == GATED, size_t, uint32_t>;
  Offset xoff[C::X_I];
#pragma unroll
  for (int j = 0; j < C::X_I; ++j) {
    const int r = (wave * C::X_I + j) * 8 + lane / P, at = min(r, rows - 1);
    Offset row = at;
    if constexpr (MODE == GATED) row = p.pairs.order[first + at] / p.pairs.top;
    xoff[j] = row * (Offset)p.k + 8 * swz16<P>(r, lane % P);
  }
  auto issue_x = [&](int t, int buffer) {
    const int k0 = begin(t);
    uint8_t* buf = lds + buffer * C::X_BYTES;
#pragma unroll
    for (int j = 0; j < C::X_I; ++j) {
      const int i = wave * C::X_I + j;
      Offset o = xoff[j];
      if (half_step(k0) && swz16<P>(i * 8 + lane / P, lane % P) >= P / 2) o -= KS / 2;
      dma16(x0 + k0 + o, buf + i * 1024);
    }
  };
  // W: this thread has half `wh` (32 values of a step) of LDS row wr.  A wave's 32 rows are neighbours (GATED: of
  // every 64 rows the first 32 are gate rows, the others their up rows).
  const int groups = p.k / G;
  constexpr int gshift = G == 32 ? 5 : G == 64 ? 6 : 7;
  const int wh = tid & 1, wr = tid / 2;
  const int col0 = min(n0 + 32 * (MODE == GATED ? wave / 2 : wave), p.n - 1);
  const uint32_t wlocal = (uint32_t)min(lane / 2, p.n - 1 - col0);
  const size_t wrow = (size_t)expert * (H * p.n) + (MODE == GATED ? (size_t)(wave % 2) * p.n : 0) + col0;
  const uint8_t* const wcode = p.w.codes + wrow * (p.k / 2);
  const uint16_t* const wscale = p.w.scales + wrow * groups;
  const uint8_t* const wzero = p.w.zeros == nullptr ? nullptr : p.w.zeros + wrow * groups;
  const uint32_t coff = wlocal * (uint32_t)(p.k / 2) + 16 * wh, soff = wlocal * (uint32_t)groups + (G == 32 ? wh : 0);
  struct Codes {
    u32x4 q;
    uint32_t s, z;
  };
  auto load_w = [&](Codes& c, int t) {
    const int k0 = begin(t);
    const uint32_t back = half_step(k0) ? wh : 0;
    c.q = *reinterpret_cast<const u32x4*>(wcode + k0 / 2 + (coff - 16 * back));
    c.s = (wscale + (k0 >> gshift))[soff - back];
    c.z = p.w.zeros == nullptr ? kInt4Zero : (wzero + (k0 >> gshift))[soff - back];
  };
  uint8_t* const wlds = lds + C::W_OFF;
  float* const mlds = reinterpret_cast<float*>(lds + C::M_OFF);
  // values 8 d .. 8 d + 7 of the thread's 32 of step t, into buffer b
  auto store_w = [&](const Codes& c, int t, int b, int d) {
    // 2^e: the exponent's bits alone (2^-126 for subnormals, whose m is below 1; Inf and NaN: Inf).  Past k and
    // with a scale of 0: values 0 whatever the codes, and m = 1.
    const bool none = t * KS + 32 * wh >= p.k || (c.s & 0x7FFFu) == 0;
    const uint32_t exponent = (c.s & 0x7F80u) << 16;
    const float s = none ? 0.0f : __uint_as_float(max(exponent, 0x00800000u));
    *reinterpret_cast<u32x4*>(wlds + b * C::W_BYTES + wr * RB + 16 * swz16<P>(wr, 4 * wh + d)) =
        widen(c.q[d], s, -(float)c.z * s);
    if (d == 0) {
      // the mantissa and the sign, in 1's binade; a subnormal's without the leading bit; NaN stays one
      const uint32_t one = (c.s & 0x807Fu) << 16 | 0x3F800000u;
      float m = __uint_as_float(one);
      if (exponent == 0) m -= __uint_as_float((c.s & 0x8000u) << 16 | 0x3F800000u);
      if (exponent == 0x7F800000u) m = (c.s & 0x7Fu) != 0 ? __builtin_nanf("") : __uint_as_float(one & 0xFF800000u);
      mlds[(b * 2 + wh) * C::BN + wr] = none ? 1.0f : m;
    }
  };

  f32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  auto fence = [] {  // the loads of W stay where they are among those of X: the waits count on it
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  Codes c[2];
  issue_x(0, 0);
  fence();
  load_w(c[0], 0);
#pragma unroll
  for (int d = 0; d < 4; ++d) store_w(c[0], 0, 0, d);
  fence();
  load_w(c[1], 1);
  fence();
  load_w(c[0], 2);
  fence();
  float unit[TJ];  // the sums are times this
#pragma unroll
  for (int j = 0; j < TJ; ++j) unit[j] = 1.0f;
  // The 32-row parts of a tile are dealt to its WM rows of waves in turn; of a tile with few rows only the first
  // LIVE parts of each are multiplied (an expert's last tile: 3 of 8 of all rows of 256-row tiles at 222 pairs an
  // expert), in code of their own, since branches around the instructions would keep them from overlapping.
  auto multiply = [&](auto live) {
    constexpr int LIVE = decltype(live)::value;
    for (int t0 = 0; t0 < steps; t0 += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // the buffers' number too
        const int t = t0 + u;
        if (t >= steps) break;
        // X of this step has arrived, everybody's part of W is written, and the other buffers are read
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        if (t < 2) wait_vmcnt<0>();  // the first loads were issued in another order
        else wait_vmcnt<2>();        // those of W behind X are two, or three with zero points
        __builtin_amdgcn_s_barrier();
        fence();
        // Rows of the parts that are multiplied alone (uniform in the wave): 64 experts of 4096 x 1792, 60 rows each, 303
        // us gated from 323 and 159 down from 173; 222 rows on average, 590 from 589 and 340 from 344.
        if (LIVE == TI || wave * C::X_I * 8 < LIVE * 32 * C::WM) issue_x(t + 1, 1 - u);
        fence();
        const uint8_t* xb = lds + u * C::X_BYTES;
        const uint8_t* wb = wlds + u * C::W_BYTES;
        bf16x8 a[2][LIVE], b[2][TJ];
        auto read = [&](int kk) {
#pragma unroll
          for (int i = 0; i < LIVE; ++i) {
            const int r = (i * C::WM + wm) * 32 + (lane & 31);
            a[kk & 1][i] = __builtin_bit_cast(
                bf16x8, *reinterpret_cast<const u32x4*>(xb + r * RB + 16 * swz16<P>(r, 2 * kk + (lane >> 5))));
          }
#pragma unroll
          for (int j = 0; j < TJ; ++j) {
            const int r = (wn * TJ + j) * 32 + (lane & 31);
            b[kk & 1][j] = __builtin_bit_cast(
                bf16x8, *reinterpret_cast<const u32x4*>(wb + r * RB + 16 * swz16<P>(r, 2 * kk + (lane >> 5))));
          }
        };
        // at the first step of a group (groups of 32: twice a step)
        auto rescale = [&](int h) {
#pragma unroll
          for (int j = 0; j < TJ; ++j) {
            const float m = mlds[(u * 2 + h) * C::BN + (wn * TJ + j) * 32 + (lane & 31)];
            const float f = unit[j] / m;
            unit[j] = m;
#pragma unroll
            for (int i = 0; i < LIVE; ++i)
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[i][j][e] *= f;
          }
        };
        read(0);
        if constexpr (G < 128) rescale(0);
        else if (u % 2 == 0) rescale(0);
#pragma unroll
        for (int kk = 0; kk < KS / 16; ++kk) {
          if (kk == 2 && G == 32) rescale(1);
          if (kk + 1 < KS / 16) read(kk + 1);  // while this one is multiplied
#pragma unroll
          for (int i = 0; i < LIVE; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[kk & 1][i], b[kk & 1][j], acc[i][j], 0, 0, 0);
          store_w(c[1 - u], t + 1, 1 - u, kk);  // past the last step: into a buffer that nobody reads
        }
        load_w(c[1 - u], t + 3);
        fence();
      }
    }
  };
  // Half of a SIMD's two waves ahead of the other: left alone they multiply and widen at the same times.
  if (C::NT == 512 && wm == 1) __builtin_amdgcn_s_setprio(1);
  if constexpr (MODE == PLAIN) {
    multiply(std::integral_constant<int, TI>());
  } else {
    const int live = (rows + 32 * C::WM - 1) / (32 * C::WM);  // uniform in the workgroup
    if constexpr (TI == 4) {
      if (live >= 4) multiply(std::integral_constant<int, 4>());
      else if (live == 3) multiply(std::integral_constant<int, 3>());
      else if (live == 2) multiply(std::integral_constant<int, 2>());
      else multiply(std::integral_constant<int, 1>());
    } else {
      if (live >= 2) multiply(std::integral_constant<int, TI>());
      else multiply(std::integral_constant<int, 1>());
    }
  }
  wait_vmcnt<0>();  // loads into LDS end before the workgroup does

#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ / H; ++j) {
      const int col = n0 + (wn * (TJ / H) + j) * 32 + (lane & 31);
      if (col >= p.n) continue;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int row = (i * C::WM + wm) * 32 + 8 * (e / 4) + 4 * (lane >> 5) + e % 4;
        if (row >= rows) continue;
        float v = acc[i][j][e] * unit[j];
        if constexpr (MODE == GATED) v = silu_mul(v, acc[i][TJ - 1][e] * unit[TJ - 1]);
        if constexpr (MODE == DOWN) p.part[(size_t)pair_of[row] * p.n + col] = v;
        else p.y[(size_t)(first + row) * p.n + col] = (uint16_t)f32x2_to_bf16x2(v, 0.0f);
      }
    }
}

template <class C, int MODE>
hipError_t launch(Args a, int64_t tiles, hipStream_t s) {
  constexpr int cols = MODE == GATED ? C::BN / 2 : C::BN;
  a.nblocks = (a.n + cols - 1) / cols;
  if (tiles * a.nblocks >= (int64_t)1 << 31) return hipErrorInvalidConfiguration;
  a.tiles = (int)tiles;
  const int64_t grid = (tiles * a.nblocks + 7) / 8 * 8;
  if (grid * C::NT >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;  // HIP counts threads in 32 bits
  const dim3 g((uint32_t)grid), block(C::NT);
  if (a.group == 128) hipLaunchKernelGGL((int4_tiled_kernel<C, MODE, 128>), g, block, 0, s, a);
  else if (a.group == 64) hipLaunchKernelGGL((int4_tiled_kernel<C, MODE, 64>), g, block, 0, s, a);
  else hipLaunchKernelGGL((int4_tiled_kernel<C, MODE, 32>), g, block, 0, s, a);
  return hipGetLastError();
}

template <int MODE, class F>
hipError_t by_size(int cfg, Args a, F tiles, hipStream_t s) {
  switch (cfg) {
    case 0: return launch<TileCfg<256, 256, 2, 4>, MODE>(a, tiles(256), s);
    case 1: return launch<TileCfg<128, 128, 2, 2>, MODE>(a, tiles(128), s);
  }
  return hipErrorInvalidConfiguration;
}

}  // namespace

hipError_t launch_int4_tiled(int cfg, const Int4Gemm& g, hipStream_t s) {
  const Args a{g.m, g.n, g.k, g.group, g.x, g.w, g.y, nullptr, Pairs{}, 0, 0};
  return by_size<PLAIN>(cfg, a, [&](int bm) { return ((int64_t)g.m + bm - 1) / bm; }, s);
}

hipError_t launch_int4_tiled_gated(int cfg, const Int4Experts& e, hipStream_t s) {
  const Args a{0, e.f, e.d, e.group, e.x, e.gu, e.h, nullptr, e.pairs, 0, 0};
  return by_size<GATED>(cfg, a, [&](int bm) { return most_tiles(e.pairs.count, e.pairs.experts, bm); }, s);
}

hipError_t launch_int4_tiled_down(int cfg, const Int4Experts& e, hipStream_t s) {
  const Args a{0, e.d, e.f, e.group, e.h, e.down, nullptr, e.part, e.pairs, 0, 0};
  return by_size<DOWN>(cfg, a, [&](int bm) { return most_tiles(e.pairs.count, e.pairs.experts, bm); }, s);
}

}  // namespace sp24
