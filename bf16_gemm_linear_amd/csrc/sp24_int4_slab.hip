// Products with integer 4-bit weights for 3 tokens to some hundreds (up to 1024 where rows of W are few or long; or
// an expert's tokens): to about 32 the weight's bytes are the time, and behind them the bytes of X that every
// workgroup takes from L2, above it W's widening for each tile of tokens.
//
// A workgroup owns `cbs` column blocks (of 16 RB rows of W; GATED: 16 gate rows and their up rows), up to
// 16 MB tokens and a slice of K.  It puts X's slice into LDS once; its waves, cbs of them along the
// columns and kp along K, then load nothing but W, straight into registers and up to S steps of 128
// values ahead: what is in flight is all of a decode step's W, and X is read from L2 once a workgroup.
// (With X in registers beside W, every wave for itself, 16 x 4096 x 14336 took 20.6 us, 8 of them for X's
// 117 MB from L2.)  The waves' sums along K are joined through LDS; where K is cut into
// slices over workgroups too, their sums go to memory in fp32 and a second kernel adds them.  All in a fixed order.
//
// v_mfma_f32_16x16x32_bf16, A = X, B = W: lane l holds row l % 16 and values 8 (l / 16) .. + 7 of a block of
// 32; accumulator register e is token 4 (l / 16) + e, W row l % 16.  A lane loads 16 bytes of codes, block
// l / 16 of its row's four; a transposition of the 4 x 4 words of lanes l, l + 16, l + 32, l + 48 (four
// register exchanges) gives it word l / 16 of every block, so each instruction covers one block of 32 and
// any group size works.  Codes become the bf16 pairs c + q - z; the sums of c x, one more instruction for all
// the workgroup's columns, are taken off behind a group's sum.  Rows past the last are the last one again; their
// outputs are not stored.
//
// 16 x 4096 x 14336 with zero points takes 11.6 to 12.5 us and 2.6 to 3.9 for the join (14.4 a call), 16 x 14336 x
// 4096 11.9; what is left over the weight's 6 is X, a launch and its end.  77 x 6144 x 4096 by groups of 32
// takes 21.2 to 22.3, of which about 12 are the vector instructions that widen W for each of five row tiles and scale a
// sum every 32 values.  Tiles of 48 tokens and more widen less and spill.  64 experts of 4096 x 1792 at 29 tokens,
// with zero points: 114 to 116 us gated (492 MB: 4.2 to 4.3 TB/s), 65 to 66 down.
#include "sp24_dma.hpp"
#include "sp24_int4.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

enum { PLAIN = 0, GATED = 1, DOWN = 2, SLICED = 3 };  // SLICED: PLAIN over a slice of K, sums to `part`

struct Args {
  int m, n, k, group;
  const uint16_t* x;
  Int4Weight w;
  uint16_t* y;
  float* part;  // DOWN: [pairs, n]; SLICED: [slices, m, n]
  Pairs pairs;
  int cbs, kp;      // waves along the columns and along K
  int slice, chunk; // values of K of a workgroup (SLICED) and of a pass; multiples of 128
  int xbytes;       // of LDS that X takes
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

constexpr int F = 4;  // scales that a thread loads at a time

// G128: a scale covers a whole step; otherwise it is applied every 32 values.  Z: with zero points.
template <int RB, int MB, int S, int MODE, bool G128, bool Z>
__global__ __launch_bounds__(1024, 4) void int4_slab_kernel(Args p) {
  constexpr int H = MODE == GATED ? 2 : 1, OB = RB / H;  // gate rows and up rows; row blocks of the output
  static_assert(OB > 0, "GATED needs a gate and an up block");
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint32_t* const sz = reinterpret_cast<uint32_t*>(lds + p.xbytes);  // scale and zero of (row, group): bf16, Int4Zeros
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = p.cbs * p.kp;
  const int cb = wave % p.cbs, kw = wave / p.cbs;
  const int cols = 16 * OB * p.cbs, nblocks = (p.n + cols - 1) / cols;
  int nb = (int)(blockIdx.x % nblocks);
  int tile = (int)(blockIdx.x / nblocks), kbegin = 0, kend = p.k, cut = 0;
  if constexpr (MODE == SLICED) {
    const int slices = (p.k + p.slice - 1) / p.slice;
    cut = tile % slices;
    tile /= slices;
    kbegin = cut * p.slice;
    kend = min(p.k, kbegin + p.slice);
  }
  int expert = 0, first = tile * 16 * MB, rows = min(16 * MB, p.m - first);
  if constexpr (MODE == GATED || MODE == DOWN)
    if (!find_tile<16 * MB>(p.pairs, (int)blockIdx.x, nblocks, lane, expert, first, rows, nb)) return;

  // Per-lane offsets are 32-bit from uniform bases (k <= 2^20, at most 16 * 16 * RB rows).
  const int half = p.k / 2, groups = p.k / p.group;
  const int gshift = p.group == 32 ? 0 : p.group == 64 ? 1 : 2;
  const int n0 = nb * cols, ncols = min(cols, p.n - n0);
  const size_t row0 = (size_t)expert * (H * p.n) + n0;
  const uint8_t* const codes = p.w.codes + row0 * half;
  const uint8_t* const codes_up = codes + (size_t)p.n * half;  // GATED
  const uint16_t* const scales = p.w.scales + row0 * groups;
  const uint16_t* const scales_up = scales + (size_t)p.n * groups;
  const uint8_t* const zeros = p.w.zeros == nullptr ? nullptr : p.w.zeros + row0 * groups;
  const uint8_t* const zeros_up = p.w.zeros == nullptr ? nullptr : zeros + (size_t)p.n * groups;
  uint32_t wrow[OB];
#pragma unroll
  for (int i = 0; i < OB; ++i) wrow[i] = (uint32_t)min(16 * (cb * OB + i) + r, ncols - 1) * (uint32_t)half;

  f32x4 acc[RB][MB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const f32x4 zero{0.f, 0.f, 0.f, 0.f};
  const Int4Bits<Z> bits;
  constexpr uint32_t all = Int4Bits<Z>::kConstant;
  const bf16x8 constant = __builtin_bit_cast(bf16x8, u32x4{all, all, all, all});

  for (int k0 = kbegin; k0 < kend; k0 += p.chunk) {
    const int kc = min(p.chunk, kend - k0);               // values of this pass
    const int blocks = kc / 32, steps = (blocks + 3) / 4;  // a last step can have fewer than four blocks
    const int pieces = 16 * steps;                         // 16-byte pieces of a row of X in LDS
    const int g0 = k0 / p.group, gc = kc / p.group;
    const int stride = gc | 1;  // odd: the rows' words lie in different banks
    // this wave's step t: pairs of steps, the kp waves in turn
    auto number = [&](int t) { return (t / 2 * p.kp + kw) * 2 + t % 2; };
    auto load = [&](u32x4 (&w)[RB], int t) {
      const int b = min(4 * min(number(t), steps - 1) + q, blocks - 1);  // this lane's block of its row's four
      const uint32_t at = (uint32_t)(k0 / 2) + 16u * (uint32_t)b;
#pragma unroll
      for (int i = 0; i < RB; ++i)
        w[i] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4*>((i < OB ? codes : codes_up) + (wrow[i % OB] + at)));
    };
    auto compute = [&](u32x4 (&wq)[RB], int t) {
      const int step = number(t);
      if (step >= steps) return;  // uniform
      const uint32_t* const szr = sz + (16 * cb * OB + r) * stride + (4 * step >> gshift);
      auto x = [&](int j, int i) {
        const int row = min(16 * j + r, rows - 1);
        const int piece = 16 * step + ((4 * i + q) ^ (row & 15));
        return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(lds + (row * pieces + piece) * 16));
      };
      // row block i's scale words: gate rows come before the workgroup's up rows
      auto both = [&](int i, int g) { return szr[(16 * (i % OB) + (i < OB ? 0 : cols)) * stride + g]; };
      bf16x8 b[RB][4];  // of every block
      float sc[RB][G128 ? 1 : 4], times[RB][G128 ? 1 : 4];  // of c x
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        uint32_t w[4] = {wq[i][0], wq[i][1], wq[i][2], wq[i][3]}, z = 0;
        transpose4(w);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          if (d == 0 || !G128) {
            // past the row's end (a last step of fewer than four blocks): unused
            const uint32_t s = both(i, G128 ? 0 : min(d >> gshift, gc - 1 - (4 * step >> gshift)));
            sc[i][d] = __uint_as_float(s & 0xFFFF0000u);
            if constexpr (Z) {
              z = Int4Zeros::bytes(s);
              times[i][d] = Int4Zeros::times(s);
            }
          }
          b[i][d] = bits.values(w[d], z);
        }
      }
      const int left = blocks - 4 * step;  // G128: at least four
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        // a group's sums of this row block's columns, and of c x
        auto add = [&](int i, int d, const f32x4& v, const f32x4& cx) {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] += sc[i][d] * (Z ? v[e] - times[i][d] * cx[e] : v[e] - cx[e]);
        };
        if constexpr (G128) {
          f32x4 v[RB], cx = zero;
#pragma unroll
          for (int i = 0; i < RB; ++i) v[i] = zero;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const bf16x8 a = x(j, d);
            cx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, constant, cx, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < RB; ++i) v[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[i][d], v[i], 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < RB; ++i) add(i, 0, v[i], cx);
        } else {
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            if (d >= left) break;  // uniform
            const bf16x8 a = x(j, d);
            const f32x4 cx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, constant, zero, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < RB; ++i)
              add(i, d, __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[i][d], zero, 0, 0, 0), cx);
          }
        }
      }
    };

    // X, a row at a time, a wave's rows wave, wave + waves, ...; pieces XOR-swizzled by row, so that the 16 rows
    // of an instruction's reads lie in different banks.  Pieces past the pass are its last one again: codes
    // past the row's end never meet them.
    if (k0 > kbegin) __syncthreads();  // the pass before is done with LDS
    for (int row = wave; row < rows; row += waves) {
      int64_t src = first + row;
      if constexpr (MODE == GATED) src = p.pairs.order[first + row] / p.pairs.top;
      const uint16_t* const xr = p.x + src * p.k + k0;
      for (int s0 = 0; s0 < pieces; s0 += 64) {
        const int slot = s0 + lane;
        if (slot < pieces) dma16(xr + 8 * min((slot & ~15) | ((slot ^ row) & 15), 4 * blocks - 1),
                                 lds + (row * pieces + s0) * 16);
      }
    }
    // The scales: up to 64 lanes along the groups, the rest of the threads along the rows (GATED: the gate
    // rows, then the up rows).
    int ashift = 6;
    while (ashift > 0 && (1 << ashift) / 2 >= gc) --ashift;
    const int per = (waves * 64) >> ashift;
    for (int g = tid & ((1 << ashift) - 1); g < gc; g += 1 << ashift) {
      for (int row = tid >> ashift; row < H * cols; row += F * per) {
        uint32_t fs[F], fz[F];
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const int at = min(row + f * per, H * cols - 1);
          const bool up = H == 2 && at >= cols;
          const uint32_t o = (uint32_t)min(up ? at - cols : at, ncols - 1) * (uint32_t)groups + (uint32_t)(g0 + g);
          fs[f] = (up ? scales_up : scales)[o];
          fz[f] = Z ? (up ? zeros_up : zeros)[o] : 0;
        }
#pragma unroll
        for (int f = 0; f < F; ++f)
          if (row + f * per < H * cols) sz[(row + f * per) * stride + g] = fs[f] << 16 | Int4Zeros::of(fz[f]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);

    const int pairs = (steps + 1) / 2;
    const int mine = pairs > kw ? (pairs - kw + p.kp - 1) / p.kp * 2 : 0;  // steps, at most one of them past the end
    u32x4 st[S][RB];
#pragma unroll
    for (int u = 0; u < S; ++u) load(st[u], u);
    __builtin_amdgcn_sched_barrier(0);
    // everybody's X and scales are there: the loads of W came last, so all but they are done
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    wait_vmcnt<S * RB>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // One copy of the code a step in flight and no more: a kernel's instructions are fetched anew at every
    // launch, and with 18 copies (6 steps in flight, the last ones unrolled apart) 16 x 14336 x 4096 took 16.1 us
    // from 12.1.  So the loads past the last step are made too, of addresses that were just read.
    for (int t = 0; t < mine; t += S) {
#pragma unroll
      for (int u = 0; u < S; ++u) {
        compute(st[u], t + u);
        __builtin_amdgcn_sched_barrier(0);
        load(st[u], t + u + S);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  __syncthreads();
  // wave (kw, cb)'s tile (i, j) at red[((kw cbs + cb) RB + i) MB + j]
  f32x4(*red)[64] = reinterpret_cast<f32x4(*)[64]>(lds);
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) red[(wave * RB + i) * MB + j][lane] = acc[i][j];
  __syncthreads();
  auto sum = [&](int at, int l) {
    f32x4 v = red[at][l];
    for (int z = 1; z < p.kp; ++z) v += red[z * p.cbs * RB * MB + at][l];
    return v;
  };
  for (int t = tid; t < p.cbs * OB * MB * 64; t += waves * 64) {
    const int l = t & 63, j = t / 64 % MB, i = t / 64 / MB % OB, c = t / 64 / MB / OB;
    const int at = (c * RB + i) * MB + j;
    f32x4 v = sum(at, l);
    if constexpr (MODE == GATED) {
      const f32x4 u = sum(at + OB * MB, l);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = silu_mul(v[e], u[e]);
    }
    const int col = 16 * (c * OB + i) + (l & 15);
    if (col >= ncols) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 16 * j + 4 * (l >> 4) + e;
      if (row >= rows) continue;
      if constexpr (MODE == DOWN) p.part[(size_t)p.pairs.order[first + row] * p.n + n0 + col] = v[e];
      else if constexpr (MODE == SLICED) p.part[((size_t)cut * p.m + first + row) * p.n + n0 + col] = v[e];
      else p.y[(size_t)(first + row) * p.n + n0 + col] = (uint16_t)f32x2_to_bf16x2(v[e], 0.0f);
    }
  }
}

// y = the sum of the slices, in their order; 1 or 4 values a thread.
template <int V>
__global__ __launch_bounds__(256) void int4_join_kernel(const float* __restrict__ part, int64_t count, int slices,
                                                        uint16_t* __restrict__ y) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
  if (at >= count) return;
  if constexpr (V == 4) {
    f32x4 v = *reinterpret_cast<const f32x4*>(part + at);
    for (int z = 1; z < slices; ++z) v += *reinterpret_cast<const f32x4*>(part + z * count + at);
    *reinterpret_cast<u32x2*>(y + at) = u32x2{f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3])};
  } else {
    float v = part[at];
    for (int z = 1; z < slices; ++z) v += part[z * count + at];
    y[at] = (uint16_t)f32x2_to_bf16x2(v, 0.0f);
  }
}

constexpr int kLds = 160 * 1024;

template <int RB, int MB, int S, int MODE>
hipError_t launch(Args a, const SlabPlan& q, int64_t tiles, hipStream_t s) {
  constexpr int H = MODE == GATED ? 2 : 1;
  const int cols = 16 * (RB / H) * q.cbs, waves = q.cbs * q.kp;
  a.cbs = q.cbs;
  a.kp = q.kp;
  a.slice = q.slice;
  a.chunk = q.chunk;
  const int rows = MODE == PLAIN || MODE == SLICED ? (a.m < 16 * MB ? a.m : 16 * MB) : 16 * MB;
  a.xbytes = rows * ((q.chunk + 127) / 128 * 256);
  const int scales = H * cols * ((q.chunk / a.group) | 1) * 4, red = waves * RB * MB * 1024;
  const int lds = a.xbytes + scales > red ? a.xbytes + scales : red;
  if (lds > kLds || waves < 1 || waves > 16) return hipErrorInvalidConfiguration;
  const int64_t grid = tiles * ((a.n + cols - 1) / cols);
  if (grid * waves * 64 >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;  // HIP counts threads in 32 bits
  const dim3 g((uint32_t)grid), block(waves * 64);
  const bool z = a.w.zeros != nullptr;
  if (a.group == 128 && z) hipLaunchKernelGGL((int4_slab_kernel<RB, MB, S, MODE, true, true>), g, block, lds, s, a);
  else if (a.group == 128) hipLaunchKernelGGL((int4_slab_kernel<RB, MB, S, MODE, true, false>), g, block, lds, s, a);
  else if (z) hipLaunchKernelGGL((int4_slab_kernel<RB, MB, S, MODE, false, true>), g, block, lds, s, a);
  else hipLaunchKernelGGL((int4_slab_kernel<RB, MB, S, MODE, false, false>), g, block, lds, s, a);
  return hipGetLastError();
}

template <int MODE>
hipError_t by_size(const Args& a, const SlabPlan& q, int64_t tiles, hipStream_t s) {
  if (q.mb == 1) return launch<2, 1, 2, MODE>(a, q, tiles, s);
  if (q.mb == 2) return launch<2, 2, 2, MODE>(a, q, tiles, s);
  return hipErrorInvalidConfiguration;
}

}  // namespace

hipError_t launch_int4_slab(const SlabPlan& q, const Int4Gemm& g, float* part, hipStream_t s) {
  Args a{g.m, g.n, g.k, g.group, g.x, g.w, g.y, part, Pairs{}, 0, 0, 0, 0, 0};
  const int64_t tiles = ((int64_t)g.m + 16 * q.mb - 1) / (16 * q.mb);
  if (q.slice >= g.k) return by_size<PLAIN>(a, q, tiles, s);
  const int slices = (g.k + q.slice - 1) / q.slice;
  const hipError_t e = by_size<SLICED>(a, q, tiles * slices, s);
  if (e != hipSuccess) return e;
  const int64_t count = (int64_t)g.m * g.n;
  if (count % 4 == 0)
    hipLaunchKernelGGL(int4_join_kernel<4>, dim3((uint32_t)((count / 4 + 255) / 256)), dim3(256), 0, s, part, count,
                       slices, g.y);
  else
    hipLaunchKernelGGL(int4_join_kernel<1>, dim3((uint32_t)((count + 255) / 256)), dim3(256), 0, s, part, count, slices,
                       g.y);
  return hipGetLastError();
}

hipError_t launch_int4_slab_gated(const SlabPlan& q, const Int4Experts& e, hipStream_t s) {
  const Args a{0, e.f, e.d, e.group, e.x, e.gu, e.h, nullptr, e.pairs, 0, 0, 0, 0, 0};
  return by_size<GATED>(a, q, most_tiles(e.pairs.count, e.pairs.experts, 16 * q.mb), s);
}

hipError_t launch_int4_slab_down(const SlabPlan& q, const Int4Experts& e, hipStream_t s) {
  const Args a{0, e.d, e.f, e.group, e.h, e.down, nullptr, e.part, e.pairs, 0, 0, 0, 0, 0};
  return by_size<DOWN>(a, q, most_tiles(e.pairs.count, e.pairs.experts, 16 * q.mb), s);
}

}  // namespace sp24
