// Products of MXFP4 operands for tens to a few thousand tokens: waves that share nothing.
//
// A workgroup owns 32 TI rows of W (gated: half of them gate rows, half their up rows) by
// 32 TJ tokens, and each of its KW waves the whole of that tile for every KW-th step of 256
// values of K.  A wave loads a step's codes and scales into LDS buffers of its own
// (global_load_lds: whole 128-byte lines of 8 rows an instruction), reads all of it into
// registers, starts the loads of its next step into the same buffer and multiplies.  So
// every byte is read from LDS once (tiles whose waves split the outputs read it two to four
// times, and at one tile a CU that is what bounds them), no wave waits for another before
// the end, and the loads of KW waves are in flight all the time.  The waves' sums are joined
// through LDS in a fixed order, a part of the tile at a time.
//
// Measured in HIP graphs, against the best tiled configuration: 4096 x 14336 with 77 tokens 11.1 us
// (22.6), with 200 15.0 (23.0) and with 1000 39.3 (44.5; 3.0 PFLOP/s), 128 x 4096 x 4096 5.4 (8.5).  Bound by
// what a CU takes in from L2: at 77 tokens 0.7 MB, 5 us at 64 bytes a cycle, beside the weight's 6.
//
// Operands: for E2M1 codes lane l of v_mfma_scale_f32_32x32x64_f8f6f4 holds row l % 32 and
// one block of 32 values (16 bytes, one scale) of half h = l / 32.  K may be permuted as
// long as both operands agree: substep s of a step takes block 2 h + s % 2 of the row's
// scale word s / 2; the two bytes of both words that a lane needs are put into one register
// (a byte permute), and the instruction's selector picks byte s of it.  Substeps 0 and 1 are
// the step's first 128 values, so a last step of 128 (k % 256 == 128) runs only those.
// Accumulator register 4 g + e of lane l is W row 8 g + 4 h + e, token l % 32.
#include <type_traits>

#include "sp24_dma.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

constexpr int KS = 256, RB = KS / 2, P = RB / 16, SW = KS / 128;  // a step: bytes, pieces, scale words of a row

enum { PLAIN = 0, GATED_BF16 = 1, GATED_MX4 = 2 };

template <int TI_, int TJ_, int KW_, int S_>
struct WaveCfg {
  static constexpr int TI = TI_, TJ = TJ_, KW = KW_, S = S_;  // S: buffers of a wave
  static constexpr int R = 32 * TI, M = 32 * TJ;
  static constexpr int W_I = R / 8, X_I = M / 8, S_I = TI + TJ, PER = W_I + X_I + S_I;  // load instructions of a step
  static constexpr int X_OFF = R * RB, S_OFF = X_OFF + M * RB, STAGE = S_OFF + (R + M) * 8;
  static constexpr int RING = KW * S * STAGE;
  static constexpr int FIT = RING / (KW * 4096);  // 32 x 32 tiles of every wave that the join holds at a time
  static_assert(RING <= 160 * 1024 && (S - 1) * PER < 64, "LDS and counter range");
};

template <int S>
__device__ __forceinline__ f32x16 mma(i32x4 a, i32x4 b, f32x16 c, int sa, int sb) {
  const i32x8 a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, S, sa, S, sb);
}

// Where a wave loads from: uniform bases, and the rows and the place in a row of its lanes.
template <class C, bool GATED>
struct WaveLoads {
  const uint8_t *w0, *w1, *x0;
  const uint32_t *ws, *xs;
  uint32_t half;      // bytes of a row
  int n0, m0, nlast, mlast, N, M, words, lane;
  uint32_t place[2];  // byte of the line that the lane loads, in even and odd instructions
  uint32_t past[2];   // 64 where that is in the step's second half

  __device__ __forceinline__ WaveLoads(const Mx4Args& p, int n0_, int m0_, int lane_)
      : half((uint32_t)p.k / 2), n0(n0_), m0(m0_), N(p.n), M(p.m), words(p.k / 128), lane(lane_) {
    w0 = p.w + (size_t)n0 * half;
    w1 = GATED ? p.w + (size_t)(p.n + n0) * half : w0;
    x0 = p.x + (size_t)m0 * half;
    ws = p.ws;
    xs = p.xs;
    nlast = p.n - 1 - n0;
    mlast = p.m - 1 - m0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      place[j] = 16 * swz16<P>(8 * j + lane / P, lane % P);
      past[j] = place[j] >= RB / 2 ? RB / 2 : 0;
    }
  }

  // Load J of step ks into buf; rows past the last are the last one again.  A step that
  // reaches past k loads its first half twice: the second copy stays unread.
  template <int J>
  __device__ __forceinline__ void issue_one(uint8_t* buf, int ks) const {
    const bool over = ks * SW + 1 >= words;  // uniform
    if constexpr (J < C::W_I) {
      constexpr int OR = GATED ? C::R / 2 : C::R, first = 8 * J % OR;
      const uint32_t row = (uint32_t)min(first + lane / P, nlast);
      const uint8_t* base = (8 * J >= OR ? w1 : w0) + (size_t)ks * RB;
      dma16(base + (__umul24(row, half) + place[J & 1] - (over ? past[J & 1] : 0)), buf + J * 1024);
    } else if constexpr (J < C::W_I + C::X_I) {
      constexpr int j = J - C::W_I;
      const uint32_t row = (uint32_t)min(8 * j + lane / P, mlast);
      dma16(x0 + (size_t)ks * RB + (__umul24(row, half) + place[j & 1] - (over ? past[j & 1] : 0)),
            buf + C::X_OFF + j * 1024);
    } else {
      constexpr int j = J - C::W_I - C::X_I;
      const int w = ks * SW, b = w / 4, width = min(4, words - 4 * b);
      const bool is_w = j < C::TI;
      constexpr int OT = GATED ? C::TI / 2 : C::TI;
      const uint32_t row = is_w ? (uint32_t)(n0 + min(32 * (j % OT) + lane / SW, nlast) + (j >= OT ? N : 0))
                                : (uint32_t)(m0 + min(32 * (j - C::TI) + lane / SW, mlast));
      const uint32_t* base =
          (is_w ? ws : xs) + (size_t)4 * (is_w ? (GATED ? 2 * N : N) : M) * b + w % 4;
      dma4(base + (row * (uint32_t)width + (over ? 0 : lane % SW)), buf + C::S_OFF + j * 256);
    }
  }
  template <int J0, int J1>
  __device__ __forceinline__ void issue(uint8_t* buf, int ks) const {
    if constexpr (J0 < J1) {
      issue_one<J0>(buf, ks);
      issue<J0 + 1, J1>(buf, ks);
    }
  }
};

template <class C>
struct WaveFrag {
  i32x4 a[C::TI][4], b[C::TJ][4];
  int sa[C::TI], sb[C::TJ];
};

// Matrix instruction T of a step (substep by substep), and after it its share of the loads.
template <class C, bool GATED, int T, int T1, bool ISSUE>
__device__ __forceinline__ void multiply(f32x16 (&acc)[C::TI][C::TJ], const WaveFrag<C>& f,
                                         const WaveLoads<C, GATED>& ld, uint8_t* buf, int ks) {
  constexpr int NM = C::TI * C::TJ, PACE = 2;  // loads per instruction: out early, yet never a queue of them
  if constexpr (T < T1) {
    constexpr int s = T / NM, i = T % NM / C::TJ, j = T % C::TJ;
    acc[i][j] = mma<s>(f.a[i][s], f.b[j][s], acc[i][j], f.sa[i], f.sb[j]);
    if constexpr (ISSUE) {
      constexpr int LAST = T == 4 * NM - 1;
      ld.template issue<(PACE * T < C::PER ? PACE * T : C::PER),
                        (LAST || PACE * (T + 1) > C::PER ? C::PER : PACE * (T + 1))>(buf, ks);
    }
    __builtin_amdgcn_sched_barrier(0);
    multiply<C, GATED, T + 1, T1, ISSUE>(acc, f, ld, buf, ks);
  }
}

template <class C, int MODE>
__global__ __launch_bounds__(C::KW * 64, C::KW / 4) void mx4_wave_kernel(Mx4Args p) {
  constexpr bool GATED = MODE == GATED_BF16 || MODE == GATED_MX4;
  constexpr int TI = C::TI, TJ = C::TJ, KW = C::KW, S = C::S;
  constexpr int OT = GATED ? TI / 2 : TI;  // row tiles of the output
  static_assert(!GATED || TI % 2 == 0, "a wave holds gate tiles and their up tiles");
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::RING];

  const int tid = threadIdx.x, lane = tid & 63;
  const int kw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r = lane & 31;

  // tile order: each XCD (workgroups b % 8) a contiguous range, in it groups of 8 tile
  // columns, so that workgroups running together share tiles in their XCD's L2
  constexpr int GROUP_N = 8;
  const int tiles_n = (p.n + 32 * OT - 1) / (32 * OT), tiles_m = (p.m + C::M - 1) / C::M, total = tiles_n * tiles_m;
  const int xcd = blockIdx.x % 8;
  const int pid = xcd * (total / 8) + min(xcd, total % 8) + (int)blockIdx.x / 8;
  const int per_group = GROUP_N * tiles_m, group = pid / per_group, first = group * GROUP_N;
  const int gsize = min(tiles_n - first, GROUP_N);
  const int n0 = (first + pid % per_group % gsize) * 32 * OT, m0 = pid % per_group / gsize * C::M;

  const int words = p.k / 128, nsteps = (p.k + KS - 1) / KS;
  const int cnt = nsteps > kw ? (nsteps - kw + KW - 1) / KW : 0;  // steps of this wave: kw + KW t
  uint8_t* const ring = lds + kw * (S * C::STAGE);

  const WaveLoads<C, GATED> ld(p, n0, m0, lane);
  f32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

#pragma unroll
  for (int t = 0; t < S; ++t)
    if (t < cnt) ld.template issue<0, C::PER>(ring + t * C::STAGE, kw + KW * t);
  // bytes 2h and 2h + 1 of a row's two words
  const uint32_t sel = h == 0 ? 0x05040100u : 0x07060302u;
  int b = 0;
  auto step = [&](int t, auto issue_tag) {
    constexpr bool ISSUE = decltype(issue_tag)::value;
    if constexpr (ISSUE) wait_vmcnt<(S - 1) * C::PER>();
    else wait_later<C::PER, S - 1>(min(cnt - 1 - t, S - 1));
    asm volatile("" ::: "memory");
    uint8_t* buf = ring + b * C::STAGE;
    b = b + 1 == S ? 0 : b + 1;
    WaveFrag<C> f;
    u32x2 ra[TI], rb[TJ];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int piece = 4 * (s >> 1) + 2 * h + (s & 1);
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int row = 32 * i + r;
        f.a[i][s] = *reinterpret_cast<const i32x4*>(buf + row * RB + 16 * swz16<P>(row, piece));
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int row = 32 * j + r;
        f.b[j][s] = *reinterpret_cast<const i32x4*>(buf + C::X_OFF + row * RB + 16 * swz16<P>(row, piece));
      }
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) ra[i] = *reinterpret_cast<const u32x2*>(buf + C::S_OFF + (32 * i + r) * 8);
#pragma unroll
    for (int j = 0; j < TJ; ++j) rb[j] = *reinterpret_cast<const u32x2*>(buf + C::S_OFF + (C::R + 32 * j + r) * 8);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the buffer is read, and may be filled again
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < TI; ++i) f.sa[i] = (int)__builtin_amdgcn_perm(ra[i][1], ra[i][0], sel);
#pragma unroll
    for (int j = 0; j < TJ; ++j) f.sb[j] = (int)__builtin_amdgcn_perm(rb[j][1], rb[j][0], sel);
    const int ks = kw + KW * t;
    if constexpr (ISSUE) {
      multiply<C, GATED, 0, 4 * TI * TJ, true>(acc, f, ld, buf, ks + KW * S);
    } else {
      multiply<C, GATED, 0, 2 * TI * TJ, false>(acc, f, ld, nullptr, 0);
      if (ks * SW + 1 < words)  // uniform: the last step can hold 128 values
        multiply<C, GATED, 2 * TI * TJ, 4 * TI * TJ, false>(acc, f, ld, nullptr, 0);
    }
  };
  const int fed = max(0, cnt - S);
  for (int t = 0; t < fed; ++t) step(t, std::true_type{});
  for (int t = fed; t < cnt; ++t) step(t, std::false_type{});

  // Join: the waves put a part of their tiles (whole output tiles: gated, a gate tile and its
  // up tile) into LDS, then each sums and stores its share of that part.
  constexpr int TPU = GATED ? 2 : 1;                    // accumulator tiles per output tile
  constexpr int UNITS = OT * TJ, PART = C::FIT / TPU < UNITS ? C::FIT / TPU : UNITS;
  static_assert(PART >= 1, "an output tile of every wave fits");
  f32x4* const red = reinterpret_cast<f32x4*>(lds);
  constexpr int WSTRIDE = PART * TPU * 4 * 64;  // of a wave, in f32x4
  auto unit_sum = [&](int u, int g) {           // registers 4 g .. 4 g + 3 of unit u's tile
    f32x4 v = red[(u * 4 + g) * 64 + lane];
#pragma unroll
    for (int z = 1; z < KW; ++z) v += red[z * WSTRIDE + (u * 4 + g) * 64 + lane];
    return v;
  };
#pragma unroll
  for (int u0 = 0; u0 < UNITS; u0 += PART) {
    __syncthreads();  // the rings, or the last part, are no longer read
#pragma unroll
    for (int u = 0; u < PART; ++u)
      if (u0 + u < UNITS) {
#pragma unroll
        for (int c = 0; c < TPU; ++c)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x16& v = acc[(u0 + u) / TJ + c * OT][(u0 + u) % TJ];
            red[kw * WSTRIDE + ((u * TPU + c) * 4 + g) * 64 + lane] =
                f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
          }
      }
    __syncthreads();
    for (int u = kw; u < PART && u0 + u < UNITS; u += KW) {
      const int i = (u0 + u) / TJ, j = (u0 + u) % TJ, n = n0 + 32 * i + 4 * h, m = m0 + 32 * j + r;
      float v[16];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 a = unit_sum(u * TPU, g);
        if constexpr (GATED) {
          const f32x4 up = unit_sum(u * TPU + 1, g);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * g + e] = silu_mul(a[e], up[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * g + e] = a[e];
        }
      }
      if constexpr (MODE == GATED_MX4) {  // n % 128 == 0: the 32 columns are one block of token m
        uint32_t key = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) key = max(key, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        key = fold_lanes<32>(key, bits_max);
        const uint32_t byte = mx4_scale_byte(key >> 23, key == 0);
        const uint32_t q0 = mx4_codes8(v, byte), q1 = mx4_codes8(v + 8, byte);
        const int nb = n0 + 32 * i;
        if (m < p.m && nb < p.n) {
          uint16_t* o = reinterpret_cast<uint16_t*>(p.hq + (size_t)m * (p.n / 2) + nb / 2) + h;
          o[0] = (uint16_t)q0;
          o[2] = (uint16_t)(q0 >> 16);
          o[4] = (uint16_t)q1;
          o[6] = (uint16_t)(q1 >> 16);
          if (h == 0)
            reinterpret_cast<uint8_t*>(p.hs + mx4_scale_word(m, nb / 128, p.m, p.n))[nb / 32 % 4] = (uint8_t)byte;
        }
      } else if (m < p.m) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = n + 8 * g;
          const bool vec = (p.n & 3) == 0 && c + 3 < p.n;
          uint16_t* y = p.y + (size_t)m * p.n + c;
          const u32x2 o{f32x2_to_bf16x2(v[4 * g], v[4 * g + 1]), f32x2_to_bf16x2(v[4 * g + 2], v[4 * g + 3])};
          if (vec) {
            *reinterpret_cast<u32x2*>(y) = o;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (c + e < p.n) y[e] = (uint16_t)(o[e / 2] >> (16 * (e & 1)));
          }
        }
      }
    }
  }
}

template <class C, int MODE>
hipError_t launch_one(const Mx4Args& a, hipStream_t s) {
  constexpr int ON = MODE == PLAIN ? C::R : C::R / 2;
  const int tiles = ((a.n + ON - 1) / ON) * ((a.m + C::M - 1) / C::M);
  hipLaunchKernelGGL((mx4_wave_kernel<C, MODE>), dim3(tiles), dim3(C::KW * 64), 0, s, a);
  return hipGetLastError();
}

template <int TI, int TJ, int KW, int S>
hipError_t launch(const Mx4Args& a, hipStream_t s) {
  using C = WaveCfg<TI, TJ, KW, S>;
  if (!a.gated) return launch_one<C, PLAIN>(a, s);
  if constexpr (TI % 2 == 0)
    return a.hq != nullptr ? launch_one<C, GATED_MX4>(a, s) : launch_one<C, GATED_BF16>(a, s);
  else
    return hipErrorInvalidConfiguration;  // never planned: a wave would hold no gate and up tile together
}

}  // namespace

hipError_t launch_mx4_wave(int cfg, const Mx4Args& a, hipStream_t s) {
  switch (cfg) {
    case 0: return launch<4, 4, 4, 1>(a, s);
    case 1: return launch<4, 2, 4, 1>(a, s);
    case 2: return launch<2, 4, 4, 1>(a, s);
    case 3: return launch<2, 2, 4, 2>(a, s);
    case 4: return launch<2, 1, 4, 3>(a, s);
    case 5: return launch<1, 2, 4, 3>(a, s);
    default: return hipErrorInvalidConfiguration;
  }
}

}  // namespace sp24
