// Products of MXFP4 operands over LDS tiles: Y[m, n] = sum_k X[m, k] W[n, k], and the
// gated product h = silu(X Wg^T) (X Wu^T) with a bf16 or MXFP4 epilogue.
//
// A workgroup owns BN rows of W (gated: BN/2 gate rows and the same BN/2 up rows) by BM
// tokens and walks K in steps of 256 values: 128 bytes of codes (whole cache lines) and
// 8 bytes of scales a row, from global memory straight into a ring of LDS buffers
// (global_load_lds), STAGES - 1 steps ahead.  Waves hold TI x TJ tiles of 32 x 32 outputs
// on v_mfma_scale_f32_32x32x64_f8f6f4, whose operands carry their E8M0 scales: no value
// is ever widened.
//
// Operands: for E2M1 codes lane l of the instruction holds row l % 32 and one block of 32
// values (16 bytes, one scale) of half h = l / 32.  K may be permuted as long as both
// operands agree: substep s of a step takes block 2 h + s % 2 of the row's scale word
// s / 2.  The two bytes of both words that a lane needs are put into one register once a
// step (a byte permute), and the instruction's selector picks byte s of it.  Substeps 0
// and 1 are the step's first 128 values, so a last step of 128 (k % 256 == 128) runs
// only those.  Accumulator register 4 g + e of lane l is W row 8 g + 4 h + e, token l % 32.
//
// LDS rows of 128 bytes are XOR-swizzled in 16-byte pieces; the swizzle is applied on
// the global side, since a load writes lane i's bytes to slot i.
//
// Measured: 8192 x 28672 x 8192 869 to 935 us over the cards (4.1 to 4.4 PFLOP/s) on 256 x 256, 1095
// to 1126 on 128 x 128: bound by power (1.6 GHz under load; the matrix instructions alone take 600 us,
// the loads alone 545) and by what each round's start and outputs leave idle.
// Gated 2047 x 14336 x 4096 132 to 148 us (128 x 128: 152 beside 148).  In one round of 256 x 256 tiles a step takes 0.9 us,
// near the instructions' own rate, and the start and the outputs' 32 MB 10 us.  Outputs go through
// LDS into whole rows: straight from the registers, half lines of many rows, 2048 x 32768 x 4096
// took 177 us against 164.
#include <type_traits>

#include "sp24_dma.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

constexpr int KS = 256;              // values of K per step
constexpr int RB = KS / 2;           // code bytes of a row per step
constexpr int P = RB / 16;           // 16-byte pieces of them
constexpr int SW = KS / 128;         // scale words of a row per step (a block of 4: two steps)
constexpr int GROUP_N = 8;           // tile columns per group in the tile order

enum { PLAIN = 0, GATED_BF16 = 1, GATED_MX4 = 2 };

// WHOLE (k % 512 == 0): scales are loaded by blocks of two steps, 16 bytes a row: those of W
// with the block's first step, those of X a step earlier, so that every step issues the same
// loads.  Otherwise the last block of the scales is narrower (its rows are not 16 bytes
// apart), and every step loads its own two words of each row: twice to four times the load
// instructions for the scales, 3-9% of the time at 8192 x 28672 x 8192.
template <int BN_, int BM_, int WN_, int WM_, int STAGES_, bool WHOLE_>
struct TileCfg {
  static constexpr int BN = BN_, BM = BM_, WN = WN_, WM = WM_, STAGES = STAGES_;
  static constexpr bool WHOLE = WHOLE_;
  static constexpr int NW = WN * WM, NT = NW * 64;
  static constexpr int TI = BN / WN / 32, TJ = BM / WM / 32;
  static constexpr int X_OFF = BN * RB, STAGE = X_OFF + BM * RB;
  static constexpr int SROW = WHOLE ? 16 : 8;  // scale bytes of a row in a buffer of scales
  // buffers of scales: those that can be read or in flight at a time (X's come a step earlier)
  static constexpr int SWBUFS = WHOLE ? STAGES / 2 + 1 : STAGES, SXBUFS = WHOLE ? (STAGES + 3) / 2 : STAGES;
  static constexpr int SW_OFF = STAGES * STAGE, SX_OFF = SW_OFF + SWBUFS * BN * SROW;
  static constexpr int RING = SX_OFF + SXBUFS * BM * SROW;
  static constexpr int YS = BN * 2 + 16;  // bytes per token of the output tile staged in LDS
  static constexpr int LDS = RING > BM * YS ? RING : BM * YS;
  // waves a SIMD holds: two, or one where four waves own the whole LDS
  static constexpr int OCC = NW >= 8 || 2 * LDS <= 160 * 1024 ? 2 : 1;
  static_assert(LDS <= 160 * 1024, "LDS budget");
  // load instructions of a wave and step: 8 rows of codes; 64 rows of a block of W's or X's
  // scales, or 32 rows of a step's of both
  static constexpr int W_I = BN / 8 / NW, X_I = BM / 8 / NW;
  static constexpr int S_ALL = WHOLE ? (BN > BM ? BN : BM) / 64 : (BN + BM) / 32, S_I = (S_ALL + NW - 1) / NW;
  static constexpr int PER = W_I + X_I + S_I;
  static_assert(W_I * 8 * NW == BN && X_I * 8 * NW == BM && BN % 64 == 0 && BM % 64 == 0, "rows split evenly");
};

// This wave's share of a step's loads.  Per-lane offsets are 32-bit from a uniform base.
template <class C, bool GATED>
struct Loads {
  const uint8_t* w0;       // first W row (gate row) of the tile
  const uint8_t* w1;       // gated: first up row
  const uint8_t* x0;
  const uint32_t *ws, *xs;
  uint32_t woff[C::W_I], xoff[C::X_I];
  uint32_t past[2];        // 64 where a lane's piece is in the step's second half (even, odd loads)
  uint32_t srow[C::S_I];   // row whose scales this lane loads (WHOLE: of W)
  uint32_t sxrow[C::S_I];  // WHOLE: of X
  int wave, lane, n0, m0, N, M, words;

  __device__ __forceinline__ Loads(const Mx4Args& p, int n0_, int m0_, int wave_, int lane_)
      : wave(wave_), lane(lane_), n0(n0_), m0(m0_), N(p.n), M(p.m) {
    const size_t half = (size_t)p.k / 2;
    words = p.k / 128;
    w0 = p.w + (size_t)n0 * half;
    w1 = GATED ? p.w + (size_t)(p.n + n0) * half : nullptr;
    x0 = p.x + (size_t)m0 * half;
    ws = p.ws;
    xs = p.xs;
#pragma unroll
    for (int j = 0; j < C::W_I; ++j) {
      const int s = (wave * C::W_I + j) * 64 + lane, row = s / P;
      woff[j] = (uint32_t)min(local_row(row), p.n - 1 - n0) * (uint32_t)half + 16 * swz16<P>(row, s % P);
    }
#pragma unroll
    for (int j = 0; j < C::X_I; ++j) {
      const int s = (wave * C::X_I + j) * 64 + lane, row = s / P;
      xoff[j] = (uint32_t)min(row, p.m - 1 - m0) * (uint32_t)half + 16 * swz16<P>(row, s % P);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) past[j] = swz16<P>(8 * j + lane / P, lane % P) >= P / 2 ? RB / 2 : 0;
#pragma unroll
    for (int j = 0; j < C::S_I; ++j) {
      if constexpr (C::WHOLE) {
        srow[j] = (uint32_t)scale_row(min(wave * C::S_I + j, C::BN / 64 - 1) * 64 + lane);
        sxrow[j] = (uint32_t)scale_row(C::BN + min(wave * C::S_I + j, C::BM / 64 - 1) * 64 + lane);
      } else {
        srow[j] = (uint32_t)scale_row(min(wave * C::S_I + j, C::S_ALL - 1) * 32 + lane / SW);
      }
    }
  }

  // Row of its operand of row `row` of BN + BM.
  __device__ __forceinline__ int scale_row(int row) const {
    if (row >= C::BN) return min(m0 + row - C::BN, M - 1);
    return min(n0 + local_row(row), N - 1) + (GATED && up_row(row) ? N : 0);
  }

  // gated: LDS rows of a wave are its gate rows, then its up rows
  static __device__ __forceinline__ bool up_row(int row) { return row % (C::BN / C::WN) >= C::BN / C::WN / 2; }
  static __device__ __forceinline__ int local_row(int row) {
    if constexpr (!GATED) return row;
    constexpr int WR = C::BN / C::WN, H = WR / 2;
    return row / WR * H + row % H;
  }

  __device__ __forceinline__ uint32_t past_half(int i) const { return i & 1 ? past[1] : past[0]; }

  // Load J of step ks.  A step that reaches past k loads its first half twice: the second
  // copy stays unread, and no load leaves its row.
  template <int J>
  __device__ __forceinline__ void issue_one(uint8_t* buf, int ks) const {
    const bool over = !C::WHOLE && ks * SW + 1 >= words;  // uniform
    if constexpr (J < C::W_I) {
      const int i = wave * C::W_I + J;  // 8 rows: all gate or all up
      const uint8_t* base = (GATED && up_row(i * 8) ? w1 : w0) + (size_t)ks * RB;
      dma16(base + (woff[J] - (over ? past_half(i) : 0)), buf + i * 1024);
    } else if constexpr (J < C::W_I + C::X_I) {
      constexpr int j = J - C::W_I;
      const int i = wave * C::X_I + j;
      const uint8_t* base = x0 + (size_t)ks * RB;
      dma16(base + (xoff[j] - (over ? past_half(i) : 0)), buf + C::X_OFF + i * 1024);
    }
  }

  // Scales of step ks.  Waves past the last instruction repeat it into its own place.
  __device__ __forceinline__ void issue_scales(uint8_t* lds, int ks) const {
    if constexpr (C::WHOLE) {
      // even: W's of the block that begins here; odd: X's of the next (past the last block its
      // own again, into a buffer that is not read any more)
      const bool x = ks & 1;
      const int b = min((ks + 1) / 2, words / 4 - 1);
      const uint32_t* const base = (x ? xs : ws) + (size_t)4 * (x ? M : GATED ? 2 * N : N) * b;
      uint8_t* const buf = lds + (x ? C::SX_OFF + (ks + 1) / 2 % C::SXBUFS * (C::BM * 16)
                                    : C::SW_OFF + ks / 2 % C::SWBUFS * (C::BN * 16));
#pragma unroll
      for (int j = 0; j < C::S_I; ++j) {
        const int i = min(wave * C::S_I + j, (x ? C::BM : C::BN) / 64 - 1);
        dma16(base + 4u * (x ? sxrow[j] : srow[j]), buf + i * 1024);
      }
    } else {
      const int w = ks * SW, b = w / 4;
      const uint32_t* const wsb = ws + (size_t)4 * (GATED ? 2 * N : N) * b + w % 4;
      const uint32_t* const xsb = xs + (size_t)4 * M * b + w % 4;
#pragma unroll
      for (int j = 0; j < C::S_I; ++j) {
        const int i = min(wave * C::S_I + j, C::S_ALL - 1);
        const bool is_w = i < C::BN / 32;
        dma4((is_w ? wsb : xsb) + (srow[j] * (uint32_t)min(4, words - 4 * b) + (w + 1 < words ? lane % SW : 0)),
             lds + (is_w ? C::SW_OFF + ks % C::SWBUFS * (C::BN * 8) + i * 256
                         : C::SX_OFF + ks % C::SXBUFS * (C::BM * 8) + (i - C::BN / 32) * 256));
      }
    }
  }

  template <int J0, int J1>
  __device__ __forceinline__ void issue(uint8_t* buf, int ks) const {
    if constexpr (J0 < J1) {
      issue_one<J0>(buf, ks);
      issue<J0 + 1, J1>(buf, ks);
    }
  }
  // LDS offsets of W's and X's scales of step ks (WHOLE: of its half of the block's 16 bytes a row)
  static __device__ __forceinline__ int w_scales_at(int ks) {
    if constexpr (C::WHOLE) return C::SW_OFF + ks / 2 % C::SWBUFS * (C::BN * 16) + ks % 2 * 8;
    return C::SW_OFF + ks % C::SWBUFS * (C::BN * 8);
  }
  static __device__ __forceinline__ int x_scales_at(int ks) {
    if constexpr (C::WHOLE) return C::SX_OFF + ks / 2 % C::SXBUFS * (C::BM * 16) + ks % 2 * 8;
    return C::SX_OFF + ks % C::SXBUFS * (C::BM * 8);
  }
};

// Operands of one substep; scale words of one step, as read and as the instruction takes them.
template <class C>
struct Frag {
  i32x4 a[C::TI], b[C::TJ];
};
template <class C>
struct Scales {
  u32x2 ra[C::TI], rb[C::TJ];
  int a[C::TI], b[C::TJ];
  // bytes 2h and 2h + 1 of both words
  __device__ __forceinline__ void pack(uint32_t sel) {
#pragma unroll
    for (int i = 0; i < C::TI; ++i) a[i] = (int)__builtin_amdgcn_perm(ra[i][1], ra[i][0], sel);
#pragma unroll
    for (int j = 0; j < C::TJ; ++j) b[j] = (int)__builtin_amdgcn_perm(rb[j][1], rb[j][0], sel);
  }
};

// LDS buffers that a phase reads, and where in the tile.
struct ReadFrom {
  const uint8_t *codes, *wscales, *xscales;
  int wn, wm, lane;
};

// Read T of substep s: A tiles, then B tiles, then (substep 0) the step's scale words.
template <class C, int T>
__device__ __forceinline__ void read_one(Frag<C>& f, Scales<C>& sc, const ReadFrom& rf, int s) {
  const int wn = rf.wn, wm = rf.wm, lane = rf.lane;
  const uint8_t* buf = rf.codes;
  const int h = lane >> 5, r = lane & 31, piece = 4 * (s >> 1) + 2 * h + (s & 1);
  if constexpr (T < C::TI) {
    const int row = wn * (C::BN / C::WN) + 32 * T + r;
    f.a[T] = *reinterpret_cast<const i32x4*>(buf + row * RB + 16 * swz16<P>(row, piece));
  } else if constexpr (T < C::TI + C::TJ) {
    constexpr int j = T - C::TI;
    const int row = wm * (C::BM / C::WM) + 32 * j + r;
    f.b[j] = *reinterpret_cast<const i32x4*>(buf + C::X_OFF + row * RB + 16 * swz16<P>(row, piece));
  } else if constexpr (T < 2 * C::TI + C::TJ) {
    constexpr int i = T - C::TI - C::TJ;
    sc.ra[i] = *reinterpret_cast<const u32x2*>(rf.wscales + (wn * (C::BN / C::WN) + 32 * i + r) * C::SROW);
  } else {
    constexpr int j = T - 2 * C::TI - C::TJ;
    sc.rb[j] = *reinterpret_cast<const u32x2*>(rf.xscales + (wm * (C::BM / C::WM) + 32 * j + r) * C::SROW);
  }
}
template <class C, int T0, int T1>
__device__ __forceinline__ void read(Frag<C>& f, Scales<C>& sc, const ReadFrom& rf, int s) {
  if constexpr (T0 < T1) {
    read_one<C, T0>(f, sc, rf, s);
    read<C, T0 + 1, T1>(f, sc, rf, s);
  }
}

template <int S>
__device__ __forceinline__ f32x16 mma(i32x4 a, i32x4 b, f32x16 c, int sa, int sb) {
  const i32x8 a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, S, sa, S, sb);
}

// Substep S's matrix instructions from `cur`, each followed by its share of the reads of
// the next substep (NR of them) and, in the last substep, of the loads of step fill_ks.
template <class C, bool GATED, int S, int T, bool ISSUE>
__device__ __forceinline__ void phase(f32x16 (&acc)[C::TI][C::TJ], const Frag<C>& cur,
                                      Frag<C>& nxt, Scales<C>& sc, const ReadFrom& rf, const Loads<C, GATED>& ld,
                                      uint8_t* fill, int fill_ks) {
  constexpr int NM = C::TI * C::TJ;
  constexpr bool LAST = S == 3;
  constexpr int NR = C::TI + C::TJ + (LAST ? C::TI + C::TJ : 0);
  constexpr int NL = ISSUE ? C::W_I + C::X_I : 0;
  // the reads go out with the first RS instructions, so the last cover their latency
  constexpr int RS = NM > 4 ? NM - 3 : NM;
  if constexpr (T < NM) {
    acc[T / C::TJ][T % C::TJ] =
        mma<S>(cur.a[T / C::TJ], cur.b[T % C::TJ], acc[T / C::TJ][T % C::TJ], sc.a[T / C::TJ], sc.b[T % C::TJ]);
    ld.template issue<T * NL / NM, (T + 1) * NL / NM>(fill, fill_ks);
    if constexpr (T < RS)
      read<C, T * NR / RS, (T + 1) * NR / RS>(nxt, sc, rf, LAST ? 0 : S + 1);
    __builtin_amdgcn_sched_barrier(0);
    phase<C, GATED, S, T + 1, ISSUE>(acc, cur, nxt, sc, rf, ld, fill, fill_ks);
  }
}

__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();        // bare: the ring's loads stay in flight
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <class C, int MODE>
__global__ __launch_bounds__(C::NT, C::OCC) void mx4_tiled_kernel(Mx4Args p) {
  constexpr bool GATED = MODE == GATED_BF16 || MODE == GATED_MX4;
  constexpr int TI = C::TI, TJ = C::TJ, ON = GATED ? C::BN / 2 : C::BN;  // output columns
  static_assert(!GATED || TI % 2 == 0, "a wave holds gate tiles and their up tiles");
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::LDS];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / C::WM, wm = wave % C::WM;

  // tile order: each XCD (workgroups b % 8) a contiguous range, in it groups of GROUP_N
  // tile columns, so that workgroups running together share tiles in their XCD's L2
  const int tiles_n = (p.n + ON - 1) / ON, tiles_m = (p.m + C::BM - 1) / C::BM, total = tiles_n * tiles_m;
  const int xcd = blockIdx.x % 8;
  const int pid = xcd * (total / 8) + min(xcd, total % 8) + (int)blockIdx.x / 8;
  const int per_group = GROUP_N * tiles_m, group = pid / per_group, first = group * GROUP_N;
  const int gsize = min(tiles_n - first, GROUP_N);
  const int n0 = (first + pid % per_group % gsize) * ON, m0 = pid % per_group / gsize * C::BM;

  f32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  // Ring: step ks in buffer ks % STAGES.  Within a step, substep s + 1 is read while
  // substep s is multiplied; before the last substep's instructions each wave waits for
  // its own loads of step ks + 1 and its reads of step ks, and the barrier then makes
  // step ks + 1 visible and frees buffer ks % STAGES for step ks + STAGES.
  constexpr int STAGES = C::STAGES, PER = C::PER;
  const int words = p.k / 128;
  const int nks = (p.k + KS - 1) / KS;
  const Loads<C, GATED> ld(p, n0, m0, wave, lane);
  if constexpr (C::WHOLE) ld.issue_scales(lds, -1);  // X's of the first block
#pragma unroll
  for (int s = 0; s < STAGES; ++s)
    if (s < nks) {
      ld.issue_scales(lds, s);
      ld.template issue<0, C::W_I + C::X_I>(lds + s * C::STAGE, s);
    }
  wait_later<PER, STAGES - 1>(min(nks - 1, STAGES - 1));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frag<C> f[2];
  Scales<C> sc;
  const uint32_t sel = lane < 32 ? 0x05040100u : 0x07060302u;  // bytes 2h and 2h + 1 of two words
  read<C, 0, 2 * (TI + TJ)>(f[0], sc, ReadFrom{lds, lds + C::SW_OFF, lds + C::SX_OFF, wn, wm, lane}, 0);

  auto wait = [] {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // this substep's operands (lgkmcnt(0))
    __builtin_amdgcn_sched_barrier(0);
  };
  int slot = 0;
  // LDS addresses are formed anew in every step: kept for every buffer of an unrolled loop
  // they cost 50 registers
  auto at = [&](int off) {
    asm volatile("" : "+s"(off));
    return lds + off;
  };
  // ISSUE: step ks + STAGES exists and is loaded here
  auto step = [&](int ks, auto issue_tag) {
    constexpr bool ISSUE = decltype(issue_tag)::value;
    uint8_t* cur = at(slot * C::STAGE);
    const ReadFrom in{cur, nullptr, nullptr, wn, wm, lane};
    slot = slot + 1 == STAGES ? 0 : slot + 1;
    wait();
    sc.pack(sel);
    phase<C, GATED, 0, 0, false>(acc, f[0], f[1], sc, in, ld, nullptr, 0);
    wait();
    phase<C, GATED, 1, 0, false>(acc, f[1], f[0], sc, in, ld, nullptr, 0);
    wait();
    phase<C, GATED, 2, 0, false>(acc, f[0], f[1], sc, in, ld, nullptr, 0);
    if constexpr (ISSUE) wait_vmcnt<(STAGES - 2) * PER>();
    else wait_later<PER, STAGES - 2>(max(0, min(nks - 2 - ks, STAGES - 2)));
    lds_barrier();
    if constexpr (ISSUE) ld.issue_scales(lds, ks + STAGES);
    // (after the last step the reads are of a valid buffer and go unused)
    phase<C, GATED, 3, 0, ISSUE>(
        acc, f[1], f[0], sc,
        ReadFrom{at(slot * C::STAGE), at(ld.w_scales_at(ks + 1)), at(ld.x_scales_at(ks + 1)), wn, wm, lane}, ld,
        cur, ks + STAGES);
  };
  const bool part = !C::WHOLE && nks * SW > words;  // the last step holds 128 values
  const int whole = part ? nks - 1 : nks, fed = max(0, nks - STAGES);
  for (int ks = 0; ks < fed; ++ks) step(ks, std::true_type{});
  for (int ks = fed; ks < whole; ++ks) step(ks, std::false_type{});
  if (part) {  // substeps 0 and 1
    const ReadFrom in{at(slot * C::STAGE), nullptr, nullptr, wn, wm, lane};
    wait();
    sc.pack(sel);
    phase<C, GATED, 0, 0, false>(acc, f[0], f[1], sc, in, ld, nullptr, 0);
    wait();
    phase<C, GATED, 1, 0, false>(acc, f[1], f[0], sc, in, ld, nullptr, 0);
  }

  const int h = lane >> 5, c = lane & 31;

  // Epilogue through LDS (the ring is free behind the barrier): the tile is staged token
  // by token and written back as rows, 16 bytes a lane.
  lds_barrier();
  constexpr int OI = GATED ? TI / 2 : TI;   // output tiles of a wave along n
  constexpr int WO = GATED ? C::BN / C::WN / 2 : C::BN / C::WN;  // output columns of a wave
  constexpr int ROWB = MODE == GATED_MX4 ? ON / 2 : ON * 2;      // bytes of a token's row
  constexpr int ROWS = ROWB + 16;                                // padded: rows spread over the banks
  static_assert(C::BM * ROWS <= C::LDS, "staged output tile fits");
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int ml = wm * (C::BM / C::WM) + 32 * j + c;
#pragma unroll
    for (int i = 0; i < OI; ++i) {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if constexpr (GATED) v[e] = silu_mul(acc[i][j][e], acc[i + TI / 2][j][e]);
        else v[e] = acc[i][j][e];
      }
      const int nl = wn * WO + 32 * i;
      if constexpr (MODE == GATED_MX4) {
        // the 32 columns are one block of token ml, half of them in lane l ^ 32
        uint32_t key = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) key = max(key, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        key = fold_lanes<32>(key, bits_max);
        const uint32_t byte = mx4_scale_byte(key >> 23, key == 0);
        const uint32_t q0 = mx4_codes8(v, byte), q1 = mx4_codes8(v + 8, byte);
        uint16_t* o = reinterpret_cast<uint16_t*>(lds + ml * ROWS + nl / 2) + h;
        o[0] = (uint16_t)q0;
        o[2] = (uint16_t)(q0 >> 16);
        o[4] = (uint16_t)q1;
        o[6] = (uint16_t)(q1 >> 16);
        const int m = m0 + ml, blk = (n0 + nl) / 32;
        if (h == 0 && m < p.m && n0 + nl < p.n)
          reinterpret_cast<uint8_t*>(p.hs + mx4_scale_word(m, blk / 4, p.m, p.n))[blk & 3] = (uint8_t)byte;
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<u32x2*>(lds + ml * ROWS + (nl + 8 * g + 4 * h) * 2) =
              u32x2{f32x2_to_bf16x2(v[4 * g], v[4 * g + 1]), f32x2_to_bf16x2(v[4 * g + 2], v[4 * g + 3])};
      }
    }
  }
  __syncthreads();
  constexpr int LPR = ROWB / 16;  // lanes per row
#pragma unroll 4
  for (int t = tid; t < C::BM * LPR; t += C::NT) {
    const int ml = t / LPR, b = t % LPR * 16, m = m0 + ml;
    const u32x4 v = *reinterpret_cast<const u32x4*>(lds + ml * ROWS + b);
    if (m >= p.m) continue;
    if constexpr (MODE == GATED_MX4) {  // n % 128 == 0: a block of 32 columns is whole or absent
      if (n0 + 2 * b < p.n) *reinterpret_cast<u32x4*>(p.hq + (size_t)m * (p.n / 2) + n0 / 2 + b) = v;
    } else {
      const int n = n0 + b / 2;
      uint16_t* yr = p.y + (size_t)m * p.n;
      if ((p.n & 7) == 0 && n + 7 < p.n) {
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(yr + n));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < p.n) yr[n + e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
      }
    }
  }
}

template <class C, int MODE>
hipError_t launch_one(const Mx4Args& a, hipStream_t s) {
  constexpr int ON = MODE == PLAIN ? C::BN : C::BN / 2;
  const int tiles = ((a.n + ON - 1) / ON) * ((a.m + C::BM - 1) / C::BM);
  hipLaunchKernelGGL((mx4_tiled_kernel<C, MODE>), dim3(tiles), dim3(C::NT), 0, s, a);
  return hipGetLastError();
}

template <int BN, int BM, int WN, int WM, int STAGES>
struct Tiles {
  template <int MODE>
  static hipError_t go(const Mx4Args& a, hipStream_t s) {
    if (a.k % 512 == 0) return launch_one<TileCfg<BN, BM, WN, WM, STAGES, true>, MODE>(a, s);
    return launch_one<TileCfg<BN, BM, WN, WM, STAGES, false>, MODE>(a, s);
  }
  static hipError_t launch(const Mx4Args& a, hipStream_t s) {
    if (!a.gated) return go<PLAIN>(a, s);
    if constexpr (BN / WN % 64 == 0)
      return a.hq != nullptr ? go<GATED_MX4>(a, s) : go<GATED_BF16>(a, s);
    else
      return hipErrorInvalidConfiguration;  // never planned: a wave would hold no gate and up tile together
  }
};

}  // namespace

hipError_t launch_mx4_tiled(int cfg, const Mx4Args& a, hipStream_t s) {
  switch (cfg) {
    case 0: return Tiles<256, 256, 2, 2, 2>::launch(a, s);
    case 1: return Tiles<256, 128, 4, 2, 2>::launch(a, s);
    case 2: return Tiles<128, 128, 2, 2, 2>::launch(a, s);
    case 3: return Tiles<128, 64, 2, 2, 3>::launch(a, s);
    case 4: return Tiles<64, 128, 2, 2, 3>::launch(a, s);
    case 5: return Tiles<64, 64, 2, 2, 3>::launch(a, s);
    default: return hipErrorInvalidConfiguration;
  }
}

}  // namespace sp24
