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
#include <type_traits>

#include "sp24_dma.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

constexpr int KS = 256;              // values of K per step
constexpr int RB = KS / 2;           // code bytes of a row per step
constexpr int P = RB / 16;           // 16-byte pieces of them
constexpr int SW = KS / 128;         // scale words of a row per step
constexpr int GROUP_N = 8;           // tile columns per group in the tile order

enum { PLAIN = 0, PARTIAL = 1, GATED_BF16 = 2, GATED_MX4 = 3 };

template <int BN_, int BM_, int WN_, int WM_, int STAGES_>
struct TileCfg {
  static constexpr int BN = BN_, BM = BM_, WN = WN_, WM = WM_, STAGES = STAGES_;
  static constexpr int NW = WN * WM, NT = NW * 64;
  static constexpr int TI = BN / WN / 32, TJ = BM / WM / 32;
  static constexpr int X_OFF = BN * RB, WS_OFF = X_OFF + BM * RB, XS_OFF = WS_OFF + BN * SW * 4;
  static constexpr int STAGE = XS_OFF + BM * SW * 4;
  static constexpr int YS = BN * 2 + 16;  // bytes per token of the output tile staged in LDS
  static constexpr int LDS = STAGES * STAGE > BM * YS ? STAGES * STAGE : BM * YS;
  static_assert(LDS <= 160 * 1024, "LDS budget");
  // load instructions of a wave per step: 8 rows of codes, or 32 rows of scales, each
  static constexpr int W_I = BN / 8 / NW, X_I = BM / 8 / NW;
  static constexpr int S_ALL = (BN + BM) / 32, S_I = (S_ALL + NW - 1) / NW;
  static constexpr int PER_STEP = W_I + X_I + S_I;
  static_assert(W_I * 8 * NW == BN && X_I * 8 * NW == BM && BN % 32 == 0 && BM % 32 == 0, "rows split evenly");
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
  int srow[C::S_I];        // row of the whole operand whose scales this lane loads
  int wave, lane, wrows, M, words;

  __device__ __forceinline__ Loads(const Mx4Args& p, int n0, int m0, int wave_, int lane_)
      : wave(wave_), lane(lane_), M(p.m) {
    const size_t half = (size_t)p.k / 2;
    wrows = GATED ? 2 * p.n : p.n;
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
      const int row = min(wave * C::S_I + j, C::S_ALL - 1) * 32 + lane / SW;  // of BN + BM
      if (row < C::BN) srow[j] = min(n0 + local_row(row), p.n - 1) + (GATED && up_row(row) ? p.n : 0);
      else srow[j] = min(m0 + row - C::BN, p.m - 1);
    }
  }

  // gated: LDS rows of a wave are its gate rows, then its up rows
  static __device__ __forceinline__ bool up_row(int row) { return row % (C::BN / C::WN) >= C::BN / C::WN / 2; }
  static __device__ __forceinline__ int local_row(int row) {
    if constexpr (!GATED) return row;
    constexpr int WR = C::BN / C::WN, H = WR / 2;
    return row / WR * H + row % H;
  }

  // Load J of step ks.  A step that reaches past k loads its first half twice: the second
  // copy stays unread, and no load leaves its row.
  template <int J>
  __device__ __forceinline__ void issue_one(uint8_t* buf, int ks) const {
    const bool over = ks * SW + 1 >= words;  // uniform
    if constexpr (J < C::W_I) {
      const int i = wave * C::W_I + J;  // 8 rows: all gate or all up
      const uint8_t* base = (GATED && up_row(i * 8) ? w1 : w0) + (size_t)ks * RB;
      dma16(base + (woff[J] - (over ? past[(C::W_I % 2 ? i : J) & 1] : 0)), buf + i * 1024);
    } else if constexpr (J < C::W_I + C::X_I) {
      constexpr int j = J - C::W_I;
      const int i = wave * C::X_I + j;
      const uint8_t* base = x0 + (size_t)ks * RB;
      dma16(base + (xoff[j] - (over ? past[(C::X_I % 2 ? i : j) & 1] : 0)), buf + C::X_OFF + i * 1024);
    } else {
      constexpr int j = J - C::W_I - C::X_I;
      // waves past the last instruction repeat it into its own place
      const int i = min(wave * C::S_I + j, C::S_ALL - 1);
      const bool is_w = i < C::BN / 32;
      const int w = ks * SW, b = w / 4, width = min(4, words - 4 * b);
      const uint32_t* base = (is_w ? ws : xs) + (size_t)4 * (is_w ? wrows : M) * b + w % 4;
      dma4(base + ((uint32_t)srow[j] * (uint32_t)width + (over ? 0 : lane % SW)), buf + C::WS_OFF + i * 256);
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

// Read T of substep s: A tiles, then B tiles, then (substep 0) the step's scale words.
template <class C, int T>
__device__ __forceinline__ void read_one(Frag<C>& f, Scales<C>& sc, const uint8_t* buf, int s, int wn, int wm,
                                         int lane) {
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
    sc.ra[i] = *reinterpret_cast<const u32x2*>(buf + C::WS_OFF + (wn * (C::BN / C::WN) + 32 * i + r) * 8);
  } else {
    constexpr int j = T - 2 * C::TI - C::TJ;
    sc.rb[j] = *reinterpret_cast<const u32x2*>(buf + C::XS_OFF + (wm * (C::BM / C::WM) + 32 * j + r) * 8);
  }
}
template <class C, int T0, int T1>
__device__ __forceinline__ void read(Frag<C>& f, Scales<C>& sc, const uint8_t* buf, int s, int wn, int wm, int lane) {
  if constexpr (T0 < T1) {
    read_one<C, T0>(f, sc, buf, s, wn, wm, lane);
    read<C, T0 + 1, T1>(f, sc, buf, s, wn, wm, lane);
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
                                      Frag<C>& nxt, Scales<C>& sc, const uint8_t* rbuf, int wn, int wm, int lane,
                                      const Loads<C, GATED>& ld, uint8_t* fill, int fill_ks) {
  constexpr int NM = C::TI * C::TJ;
  constexpr bool LAST = S == P / 2 - 1;
  constexpr int NR = C::TI + C::TJ + (LAST ? C::TI + C::TJ : 0);
  constexpr int NL = ISSUE ? C::PER_STEP : 0;
  // the reads go out with the first RS instructions, so the last cover their latency
  constexpr int RS = NM > 4 ? NM - 3 : NM;
  if constexpr (T < NM) {
    acc[T / C::TJ][T % C::TJ] =
        mma<S>(cur.a[T / C::TJ], cur.b[T % C::TJ], acc[T / C::TJ][T % C::TJ], sc.a[T / C::TJ], sc.b[T % C::TJ]);
    ld.template issue<T * NL / NM, (T + 1) * NL / NM>(fill, fill_ks);
    if constexpr (T < RS)
      read<C, T * NR / RS, (T + 1) * NR / RS>(nxt, sc, rbuf, LAST ? 0 : S + 1, wn, wm, lane);
    __builtin_amdgcn_sched_barrier(0);
    phase<C, GATED, S, T + 1, ISSUE>(acc, cur, nxt, sc, rbuf, wn, wm, lane, ld, fill, fill_ks);
  }
}

__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();        // bare: the ring's loads stay in flight
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// slice_steps: K steps of a slice (blockIdx.y), PARTIAL only.
template <class C, int MODE>
__global__ __launch_bounds__(C::NT, 2) void mx4_tiled_kernel(Mx4Args p, int slice_steps) {
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
  constexpr int STAGES = C::STAGES, PER = C::PER_STEP;
  const int all_steps = (p.k + KS - 1) / KS;
  const int words = p.k / 128;
  const int k0 = MODE == PARTIAL ? (int)blockIdx.y * slice_steps : 0;
  const int nks = MODE == PARTIAL ? min(slice_steps, all_steps - k0) : all_steps;
  const Loads<C, GATED> ld(p, n0, m0, wave, lane);
#pragma unroll
  for (int s = 0; s < STAGES; ++s)
    if (s < nks) ld.template issue<0, PER>(lds + s * C::STAGE, k0 + s);
  wait_later<PER, STAGES - 1>(min(nks - 1, STAGES - 1));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frag<C> f[2];
  Scales<C> sc;
  const uint32_t sel = lane < 32 ? 0x05040100u : 0x07060302u;
  read<C, 0, 2 * (TI + TJ)>(f[0], sc, lds, 0, wn, wm, lane);

  auto wait = [] {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // this substep's operands (lgkmcnt(0))
    __builtin_amdgcn_sched_barrier(0);
  };
  int slot = 0;
  auto first_half = [&] {
    const uint8_t* cur = lds + slot * C::STAGE;
    wait();
    sc.pack(sel);
    phase<C, GATED, 0, 0, false>(acc, f[0], f[1], sc, cur, wn, wm, lane, ld, nullptr, 0);
    wait();
    phase<C, GATED, 1, 0, false>(acc, f[1], f[0], sc, cur, wn, wm, lane, ld, nullptr, 0);
  };
  auto step = [&](int ks, auto issue_tag) {
    constexpr bool ISSUE = decltype(issue_tag)::value;
    uint8_t* cur = lds + slot * C::STAGE;
    first_half();
    slot = slot + 1 == STAGES ? 0 : slot + 1;
    wait();
    phase<C, GATED, 2, 0, false>(acc, f[0], f[1], sc, cur, wn, wm, lane, ld, nullptr, 0);
    if constexpr (ISSUE) wait_vmcnt<(STAGES - 2) * PER>();
    else wait_later<PER, STAGES - 2>(max(0, min(nks - 2 - ks, STAGES - 2)));
    lds_barrier();
    // (after the last step the reads are of a valid buffer and go unused)
    phase<C, GATED, 3, 0, ISSUE>(acc, f[1], f[0], sc, lds + slot * C::STAGE, wn, wm, lane, ld, cur, k0 + ks + STAGES);
  };
  const bool part = (k0 + nks) * SW > words;  // the last step holds 128 values
  const int whole = part ? nks - 1 : nks, fed = max(0, nks - STAGES);
  for (int ks = 0; ks < fed; ++ks) step(ks, std::true_type{});
  for (int ks = fed; ks < whole; ++ks) step(ks, std::false_type{});
  if (part) first_half();

  const int h = lane >> 5, c = lane & 31;
  if constexpr (MODE == PARTIAL) {
    float* pz = p.partial + (size_t)blockIdx.y * p.m * p.n;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int m = m0 + wm * (C::BM / C::WM) + 32 * j + c;
      if (m >= p.m) continue;
      float* pr = pz + (size_t)m * p.n;
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int n = n0 + wn * (C::BN / C::WN) + 32 * i + 8 * g + 4 * h;
          const f32x4 v = f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
          if ((p.n & 3) == 0 && n + 3 < p.n) {
            *reinterpret_cast<f32x4*>(pr + n) = v;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n + e < p.n) pr[n + e] = v[e];
          }
        }
    }
    return;
  }

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
        key = max(key, (uint32_t)__shfl_xor((int)key, 32, 64));
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
hipError_t launch(const Mx4Args& a, int split, hipStream_t s) {
  constexpr int ON = MODE == GATED_BF16 || MODE == GATED_MX4 ? C::BN / 2 : C::BN;
  const int tiles = ((a.n + ON - 1) / ON) * ((a.m + C::BM - 1) / C::BM), steps = (a.k + KS - 1) / KS;
  hipLaunchKernelGGL((mx4_tiled_kernel<C, MODE>), dim3(tiles, split), dim3(C::NT), 0, s, a, (steps + split - 1) / split);
  return hipGetLastError();
}

using Big = TileCfg<256, 256, 2, 4, 2>;
using Mid = TileCfg<128, 128, 2, 2, 2>;
using Low = TileCfg<128, 64, 2, 2, 3>;

template <class C>
hipError_t launch_mode(const Mx4Args& a, int split, hipStream_t s) {
  if (a.gated) return a.hq != nullptr ? launch<C, GATED_MX4>(a, 1, s) : launch<C, GATED_BF16>(a, 1, s);
  if (split <= 1) return launch<C, PLAIN>(a, 1, s);
  if (const hipError_t e = launch<C, PARTIAL>(a, split, s)) return e;
  GemmArgs r{};  // the reduction of the 2:4 products, without scales
  r.dtype = SP24_BF16;
  r.m = a.m;
  r.n = a.n;
  r.k = a.k;
  r.y = a.y;
  r.partial = a.partial;
  return launch_splitk_reduce(r, split, s);
}

}  // namespace

hipError_t launch_mx4_tiled(int cfg, int split, const Mx4Args& a, hipStream_t s) {
  switch (cfg) {
    case 0: return launch_mode<Big>(a, split, s);
    case 1: return launch_mode<Mid>(a, split, s);
    default: return launch_mode<Low>(a, split, s);
  }
}

}  // namespace sp24
