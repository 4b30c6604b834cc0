// Products of MXFP4 operands for few tokens (decode): the weight's bytes are the time.
//
// A workgroup owns up to 16 RBK rows of W (gated: half of them gate rows, half their up
// rows) and all of K.  Its KW waves take turns at steps of 256 values and never wait for
// each other: each wave has its own ring of S buffers in LDS, loads a step of W, X and
// their scales straight into it (global_load_lds: whole 128-byte lines of 8 rows an
// instruction), S - 1 steps ahead, and waits only for its own loads.  The rings together
// hold most of a decode step's share of W in flight, which is what hides the latency, and
// a wave's chain of waits is 1 / KW of the steps.  The waves' sums are joined through LDS
// in a fixed order.  W is read once, with the non-temporal hint; X comes from L2.
//
// Measured, calls in a row: one token 14336 x 4096 6.5 us (4.8 TB/s), gated 11.9 (5.2 TB/s, three
// weights in turn partly from the last-level cache); in HIP graphs one token 7.1 (the best of the
// other kernels 7.4), 16 tokens gated 14336 x 4096 with MXFP4 output 12.7 and 4096 x 14336 7.5 (9.8).  Bound by memory and by the first
// loads' latency; with W loaded straight into registers, less of it in flight, one token
// 14336 x 4096 took 9.2 (the rings, at first: 7.4).
//
// v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds row l % 16 (A: W, B: X) and block l / 16
// of the unit's four, so its scale is byte l / 16 of the row's word; accumulator register e
// is W row 4 (l / 16) + e, token l % 16.  Rows past the last are the last one again, and
// where fewer than 16 tokens are loaded (XR = 8) they stand for the others: their outputs
// are not stored.
#include "sp24_dma.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

enum { PLAIN = 0, GATED_BF16 = 1, GATED_MX4 = 2 };

constexpr int KS = 256, RB = KS / 2, P = RB / 16, SW = KS / 128;  // a step: bytes, pieces, scale words of a row

template <int RBK_, int MB_, int XR_, int KW_, int S_>
struct StreamCfg {
  static constexpr int RBK = RBK_, MB = MB_, XR = XR_, KW = KW_, S = S_;
  static constexpr int R = 16 * RBK;
  static constexpr int W_I = R / 8, X_I = XR / 8, S_I = (R + XR + 31) / 32;  // load instructions of a step
  static constexpr int PER = W_I + X_I + S_I;
  static constexpr int X_OFF = R * RB, S_OFF = X_OFF + XR * RB, STAGE = S_OFF + S_I * 256;
  static constexpr int RED = KW * RBK * MB * 1024;
  static constexpr int LDS = KW * S * STAGE > RED ? KW * S * STAGE : RED;
  static_assert(LDS <= 160 * 1024 && (S - 1) * PER < 64, "LDS and counter range");
  static_assert(XR % 8 == 0 && XR <= 16 * MB && (XR == 16 * MB || XR == 8), "token rows");
};

// rows: output columns of a workgroup (a multiple of 4; of 32 for GATED_MX4).
template <class C, int MODE>
__global__ __launch_bounds__(C::KW * 64, C::KW / 4) void mx4_stream_kernel(Mx4Args p, int rows) {
  constexpr bool GATED = MODE != PLAIN;
  constexpr int RBK = C::RBK, MB = C::MB, KW = C::KW, S = C::S;
  constexpr int OB = GATED ? RBK / 2 : RBK;  // row blocks of the output
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::LDS];

  const int tid = threadIdx.x, lane = tid & 63;
  const int kw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * rows, nrows = min(rows, p.n - n0);
  const int m0 = blockIdx.y * 16 * MB, mrows = min(16 * MB, p.m - m0);
  const size_t half = (size_t)p.k / 2;
  const int words = p.k / 128, nsteps = (words + SW - 1) / SW;
  const int wrows = GATED ? 2 * p.n : p.n;
  uint8_t* ring = lds + kw * (S * C::STAGE);

  // per-lane offsets of this wave's loads from uniform bases; LDS row i of W is output
  // column i % (16 OB) of the gate (i < 16 OB) or up half
  const uint8_t* const w0 = p.w + (size_t)n0 * half;
  const uint8_t* const w1 = GATED ? p.w + (size_t)(p.n + n0) * half : w0;
  const uint8_t* const x0 = p.x + (size_t)m0 * half;
  uint32_t woff[C::W_I], xoff[C::X_I], past[2];
  int srow[C::S_I];
#pragma unroll
  for (int j = 0; j < C::W_I; ++j) {
    const int row = 8 * j + lane / P;
    woff[j] = (uint32_t)min(row % (16 * OB), nrows - 1) * (uint32_t)half + 16 * swz16<P>(row, lane % P);
  }
#pragma unroll
  for (int j = 0; j < C::X_I; ++j) {
    const int row = 8 * j + lane / P;
    xoff[j] = (uint32_t)min(row, mrows - 1) * (uint32_t)half + 16 * swz16<P>(row, lane % P);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) past[j] = swz16<P>(8 * j + lane / P, lane % P) >= P / 2 ? RB / 2 : 0;
#pragma unroll
  for (int j = 0; j < C::S_I; ++j) {
    const int row = min(32 * j + lane / SW, C::R + C::XR - 1);
    srow[j] = row < C::R ? n0 + min(row % (16 * OB), nrows - 1) + (row >= 16 * OB ? p.n : 0)
                         : m0 + min(row - C::R, mrows - 1);
  }

  // Step ks into buffer b.  A step that reaches past k loads its first half twice: the
  // second copy stays unread, and no load leaves its row.
  auto issue = [&](int b, int ks) {
    uint8_t* buf = ring + b * C::STAGE;
    const bool over = ks * SW + 1 >= words;  // uniform
    const int w = ks * SW, blk = w / 4, width = min(4, words - 4 * blk);
#pragma unroll
    for (int j = 0; j < C::W_I; ++j)
      dma16_nt((j < 2 * OB ? w0 : w1) + (size_t)ks * RB + (woff[j] - (over ? past[j & 1] : 0)), buf + j * 1024);
#pragma unroll
    for (int j = 0; j < C::X_I; ++j)
      dma16(x0 + (size_t)ks * RB + (xoff[j] - (over ? past[j & 1] : 0)), buf + C::X_OFF + j * 1024);
#pragma unroll
    for (int j = 0; j < C::S_I; ++j) {
      const uint32_t* ws = p.ws + (size_t)4 * wrows * blk + w % 4;
      const uint32_t* xs = p.xs + (size_t)4 * p.m * blk + w % 4;
      // an instruction can hold rows of both operands
      const uint32_t* base = 32 * j + 31 < C::R ? ws : 32 * j >= C::R ? xs : 32 * j + lane / SW < C::R ? ws : xs;
      dma4(base + ((uint32_t)srow[j] * (uint32_t)width + (over ? 0 : lane % SW)), buf + C::S_OFF + j * 256);
    }
  };

  f32x4 acc[RBK][MB];
#pragma unroll
  for (int i = 0; i < RBK; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int cnt = nsteps > kw ? (nsteps - kw + KW - 1) / KW : 0;  // steps of this wave: kw + KW t
#pragma unroll
  for (int t = 0; t < S; ++t)
    if (t < cnt) issue(t, kw + KW * t);
  int b = 0;
  for (int t = 0; t < cnt; ++t) {
    wait_later<C::PER, S - 1>(min(cnt - 1 - t, S - 1));
    asm volatile("" ::: "memory");
    const uint8_t* buf = ring + b * C::STAGE;
    i32x4 a[RBK][SW], x[MB][SW];
    int sa[RBK][SW], sx[MB][SW];
#pragma unroll
    for (int u = 0; u < SW; ++u) {
#pragma unroll
      for (int i = 0; i < RBK; ++i) {
        const int row = 16 * i + r;
        a[i][u] = *reinterpret_cast<const i32x4*>(buf + row * RB + 16 * swz16<P>(row, 4 * u + q));
        sa[i][u] = buf[C::S_OFF + row * 8 + 4 * u + q];
      }
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const int row = (16 * j + r) % C::XR;
        x[j][u] = *reinterpret_cast<const i32x4*>(buf + C::X_OFF + row * RB + 16 * swz16<P>(row, 4 * u + q));
        sx[j][u] = buf[C::S_OFF + (C::R + row) * 8 + 4 * u + q];
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the buffer is read, and may be filled again
    __builtin_amdgcn_sched_barrier(0);
    const int ks = kw + KW * t;
    if (t + S < cnt) issue(b, ks + KW * S);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < SW; ++u) {
      if (u > 0 && ks * SW + u >= words) break;  // uniform: the last step holds 128 values
#pragma unroll
      for (int i = 0; i < RBK; ++i) {
        const i32x8 a8 = __builtin_shufflevector(a[i][u], a[i][u], 0, 1, 2, 3, -1, -1, -1, -1);
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          const i32x8 x8 = __builtin_shufflevector(x[j][u], x[j][u], 0, 1, 2, 3, -1, -1, -1, -1);
          acc[i][j] =
              __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, x8, acc[i][j], 4, 4, 0, sa[i][u], 0, sx[j][u]);
        }
      }
    }
    b = b + 1 == S ? 0 : b + 1;
  }

  // the rings are free behind the barrier; tile (i, j) of wave kw at red[kw][i MB + j]
  f32x4(*red)[RBK * MB][64] = reinterpret_cast<f32x4(*)[RBK * MB][64]>(lds);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RBK; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) red[kw][i * MB + j][lane] = acc[i][j];
  __syncthreads();
  auto sum = [&](int tile, int l) {
    f32x4 v = red[0][tile][l];
#pragma unroll
    for (int z = 1; z < KW; ++z) v += red[z][tile][l];
    return v;
  };

  if constexpr (MODE == GATED_MX4) {
    // two row blocks of 16 are one block of 32 columns: a lane takes 4 columns of each
    for (int t = tid; t < OB / 2 * MB * 64; t += KW * 64) {
      const int l = t & 63, j = t / 64 % MB, blk = t / 64 / MB;
      float v[8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const f32x4 g = sum((2 * blk + c) * MB + j, l), u = sum((2 * blk + c + OB) * MB + j, l);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * c + e] = silu_mul(g[e], u[e]);
      }
      uint32_t key = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) key = max(key, __float_as_uint(v[e]) & 0x7FFFFFFFu);
      key = fold_lanes<32>(fold_lanes<16>(key, bits_max), bits_max);
      const uint32_t byte = mx4_scale_byte(key >> 23, key == 0), c8 = mx4_codes8(v, byte);
      const int m = m0 + 16 * j + (l & 15), n = n0 + 32 * blk, qq = l >> 4;
      if (m >= p.m || 32 * blk >= nrows) continue;  // rows past the range are the next workgroup's
      uint16_t* o = reinterpret_cast<uint16_t*>(p.hq + (size_t)m * (p.n / 2) + n / 2) + qq;
      o[0] = (uint16_t)c8;
      o[4] = (uint16_t)(c8 >> 16);
      if (qq == 0)
        reinterpret_cast<uint8_t*>(p.hs + mx4_scale_word(m, n / 128, p.m, p.n))[n / 32 % 4] = (uint8_t)byte;
    }
  } else {
    for (int t = tid; t < OB * MB * 64; t += KW * 64) {
      const int l = t & 63, j = t / 64 % MB, i = t / 64 / MB;
      f32x4 v = sum(i * MB + j, l);
      if constexpr (GATED) {
        const f32x4 u = sum((i + OB) * MB + j, l);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = silu_mul(v[e], u[e]);
      }
      const int m = m0 + 16 * j + (l & 15), nl = 16 * i + 4 * (l >> 4);
      if (m >= p.m || nl >= nrows) continue;
      uint16_t* yr = p.y + (size_t)m * p.n + n0 + nl;
      const u32x2 o{f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3])};
      if ((p.n & 3) == 0) {  // then nl + 3 < nrows
        *reinterpret_cast<u32x2*>(yr) = o;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (nl + e < nrows) yr[e] = (uint16_t)(o[e / 2] >> (16 * (e & 1)));
      }
    }
  }
}

template <int RBK, int MB, int XR, int KW, int S>
hipError_t launch(const Mx4Args& a, int rows, hipStream_t s) {
  using C = StreamCfg<RBK, MB, XR, KW, S>;
  const dim3 grid((a.n + rows - 1) / rows, (a.m + 16 * MB - 1) / (16 * MB));
  if (!a.gated) {
    hipLaunchKernelGGL((mx4_stream_kernel<C, PLAIN>), grid, dim3(KW * 64), 0, s, a, rows);
    return hipGetLastError();
  }
  if (a.hq == nullptr) {
    if constexpr (RBK % 2 == 0) {
      hipLaunchKernelGGL((mx4_stream_kernel<C, GATED_BF16>), grid, dim3(KW * 64), 0, s, a, rows);
      return hipGetLastError();
    }
  } else if constexpr (RBK % 4 == 0) {
    hipLaunchKernelGGL((mx4_stream_kernel<C, GATED_MX4>), grid, dim3(KW * 64), 0, s, a, rows);
    return hipGetLastError();
  }
  return hipErrorInvalidConfiguration;  // never planned: too few row blocks for this output
}

}  // namespace

hipError_t launch_mx4_stream(int rb, int rows, const Mx4Args& a, hipStream_t s) {
  const int mb = a.m <= 8 ? 0 : a.m <= 16 ? 1 : a.m <= 32 ? 2 : 4;
  switch (10 * rb + mb) {
    case 10: return launch<1, 1, 8, 8, 4>(a, rows, s);
    case 11: return launch<1, 1, 16, 8, 4>(a, rows, s);
    case 12: return launch<1, 2, 32, 8, 2>(a, rows, s);
    case 14: return launch<1, 4, 64, 4, 3>(a, rows, s);
    case 20: return launch<2, 1, 8, 8, 3>(a, rows, s);
    case 21: return launch<2, 1, 16, 8, 2>(a, rows, s);
    case 22: return launch<2, 2, 32, 8, 2>(a, rows, s);
    case 24: return launch<2, 4, 64, 4, 3>(a, rows, s);
    case 40: return launch<4, 1, 8, 8, 2>(a, rows, s);
    case 41: return launch<4, 1, 16, 4, 3>(a, rows, s);
    case 42: return launch<4, 2, 32, 4, 3>(a, rows, s);
    case 44: return launch<4, 4, 64, 4, 2>(a, rows, s);
    case 80: return launch<8, 1, 8, 4, 2>(a, rows, s);
    case 81: return launch<8, 1, 16, 4, 2>(a, rows, s);
    default: return hipErrorInvalidConfiguration;
  }
}

}  // namespace sp24
