// Products of MXFP4 operands for few tokens (decode): the weight's bytes are the time.
//
// A workgroup owns up to 16 RBK rows of W (gated: half of them gate rows, half their up
// rows) and all of K, split over its KW waves in steps of U units of 128 values; the waves' sums are
// joined through LDS in a fixed order.  Codes go from memory straight into registers, 1 KB
// an instruction (16 rows x 64 contiguous bytes), D steps ahead: at the sizes of a decode
// step that is most of the workgroup's share of W in flight at once, which is what hides
// the latency.  W is read once, with the non-temporal hint; X comes from L2.
//
// v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds row l % 16 (A: W, B: X) and block l / 16
// of the unit's four, so its scale is byte l / 16 of the row's word; accumulator register e
// is W row 4 (l / 16) + e, token l % 16.  Rows and units that do not exist read as zero
// codes through the buffer's range check (no memory is touched); their scales are those of
// a row or unit that does exist, so a product with them is 0, and NaN only where the row's
// own result is.
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

enum { PLAIN = 0, GATED_BF16 = 2, GATED_MX4 = 3 };

constexpr int kNonTemporal = 2;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, size_t bytes) {
  const uint32_t n = bytes < 0x7FFFFFF0u ? (uint32_t)bytes : 0x7FFFFFF0u;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)n, 0x00020000);
}

// One step: U units of 128 values, codes and scale words of the wave's row and token blocks.
template <int RBK, int MB, int U>
struct Step {
  i32x4 w[RBK][U], x[MB][U];
  uint32_t ws[RBK][U], xs[MB][U];
};

// rows: output columns of a workgroup (a multiple of 4; of 32 for GATED_MX4).
template <int RBK, int MB, int KW, int U, int D, int MODE>
__global__ __launch_bounds__(KW * 64) void mx4_stream_kernel(Mx4Args p, int rows) {
  constexpr bool GATED = MODE != PLAIN;
  constexpr int OB = GATED ? RBK / 2 : RBK;  // row blocks of the output
  __shared__ __attribute__((aligned(16))) f32x4 red[KW][RBK * MB][64];

  const int tid = threadIdx.x, lane = tid & 63;
  const int kw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * rows, nrows = min(rows, p.n - n0);
  const int m0 = blockIdx.y * 16 * MB, mrows = min(16 * MB, p.m - m0);
  const size_t half = (size_t)p.k / 2;
  const int words = p.k / 128, nsteps = (words + U - 1) / U;
  const int wrows = GATED ? 2 * p.n : p.n;

  // rows past the range (rows need not be a multiple of 16) are past the buffer's end
  const __amdgpu_buffer_rsrc_t wb0 = buffer(p.w + (size_t)n0 * half, nrows * half);
  const __amdgpu_buffer_rsrc_t wb1 = GATED ? buffer(p.w + (size_t)(p.n + n0) * half, nrows * half) : wb0;
  const __amdgpu_buffer_rsrc_t xb = buffer(p.x + (size_t)m0 * half, mrows * half);
  uint32_t woff[OB], xoff[MB];
  int wsr[RBK], xsr[MB];
#pragma unroll
  for (int i = 0; i < OB; ++i) woff[i] = (uint32_t)(16 * i + r) * (uint32_t)half + 16 * q;
#pragma unroll
  for (int i = 0; i < RBK; ++i)
    wsr[i] = n0 + min(16 * (i % OB) + r, nrows - 1) + (i >= OB ? p.n : 0);
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    xoff[j] = (uint32_t)(16 * j + r) * (uint32_t)half + 16 * q;
    xsr[j] = m0 + min(16 * j + r, mrows - 1);
  }

  f32x4 acc[RBK][MB];
#pragma unroll
  for (int i = 0; i < RBK; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // step t of this wave: units U (kw + KW t) and the next
  auto load = [&](Step<RBK, MB, U>& s, int t) {
    const int step = kw + KW * t;
    uint32_t k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) k[u] = U * step + u < words ? (uint32_t)(U * step + u) * 64u : 0x80000000u;
    const int w = U * min(step, nsteps - 1), b = w / 4, width = min(4, words - 4 * b);
    const bool both = w + 1 < words;
    auto scales = [&](const uint32_t* base, int rows_all, const int* row, auto* out, int count) {
      const __amdgpu_buffer_rsrc_t sb = buffer(base + (size_t)4 * rows_all * b, (size_t)rows_all * width * 4);
#pragma unroll
      for (int i = 0; i < count; ++i) {
        const uint32_t off = ((uint32_t)row[i] * (uint32_t)width + w % 4) * 4u;
        if constexpr (U == 2) {  // a row's last word alone: the second is another row's, or past the end
          const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(sb, off, 0, 0));
          out[i][0] = v[0];
          out[i][1] = both ? v[1] : v[0];
        } else {
          out[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_raw_buffer_load_b32(sb, off, 0, 0));
        }
      }
    };
#pragma unroll
    for (int i = 0; i < RBK; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u)
        s.w[i][u] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  i < OB ? wb0 : wb1, k[u] + woff[i % OB], 0, kNonTemporal));
    scales(p.ws, wrows, wsr, s.ws, RBK);
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int u = 0; u < U; ++u)
        s.x[j][u] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(xb, k[u] + xoff[j], 0, 0));
    scales(p.xs, p.m, xsr, s.xs, MB);
  };
  auto compute = [&](const Step<RBK, MB, U>& s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int sx[MB];
#pragma unroll
      for (int j = 0; j < MB; ++j) sx[j] = (int)(s.xs[j][u] >> (8 * q));
#pragma unroll
      for (int i = 0; i < RBK; ++i) {
        const int sw = (int)(s.ws[i][u] >> (8 * q));
        const i32x8 a = __builtin_shufflevector(s.w[i][u], s.w[i][u], 0, 1, 2, 3, -1, -1, -1, -1);
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          const i32x8 b = __builtin_shufflevector(s.x[j][u], s.x[j][u], 0, 1, 2, 3, -1, -1, -1, -1);
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[i][j], 4, 4, 0, sw, 0, sx[j]);
        }
      }
    }
  };

  const int cnt = (nsteps - kw + KW - 1) / KW;  // steps of this wave (0 where nsteps <= kw)
  Step<RBK, MB, U> st[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load(st[d], d);
  for (int t = 0; t + D < cnt; t += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      compute(st[d]);
      load(st[d], t + d + D);
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d) compute(st[d]);

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
      key = max(key, (uint32_t)__shfl_xor((int)key, 16, 64));
      key = max(key, (uint32_t)__shfl_xor((int)key, 32, 64));
      const uint32_t byte = mx4_scale_byte(key >> 23, key == 0), c8 = mx4_codes8(v, byte);
      const int m = m0 + 16 * j + (l & 15), n = n0 + 32 * blk, qq = l >> 4;
      if (m >= p.m || n >= p.n) continue;
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

template <int RBK, int MB, int KW, int U, int D>
hipError_t launch(const Mx4Args& a, int rows, hipStream_t s) {
  const dim3 grid((a.n + rows - 1) / rows, (a.m + 16 * MB - 1) / (16 * MB));
  if (!a.gated) {
    hipLaunchKernelGGL((mx4_stream_kernel<RBK, MB, KW, U, D, PLAIN>), grid, dim3(KW * 64), 0, s, a, rows);
  } else if constexpr (RBK % 2 == 0) {
    if (a.hq == nullptr) {
      hipLaunchKernelGGL((mx4_stream_kernel<RBK, MB, KW, U, D, GATED_BF16>), grid, dim3(KW * 64), 0, s, a, rows);
    } else if constexpr (RBK == 4) {
      hipLaunchKernelGGL((mx4_stream_kernel<RBK, MB, KW, U, D, GATED_MX4>), grid, dim3(KW * 64), 0, s, a, rows);
    }
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_stream(int rb, int rows, const Mx4Args& a, hipStream_t s) {
  const int mb = a.m <= 16 ? 1 : a.m <= 32 ? 2 : 4;
  switch (10 * rb + mb) {
    case 11: return launch<1, 1, 8, 2, 4>(a, rows, s);
    case 12: return launch<1, 2, 8, 2, 3>(a, rows, s);
    case 14: return launch<1, 4, 8, 1, 4>(a, rows, s);
    case 21: return launch<2, 1, 8, 2, 2>(a, rows, s);
    case 22: return launch<2, 2, 8, 2, 2>(a, rows, s);
    case 24: return launch<2, 4, 8, 1, 3>(a, rows, s);
    case 41: return launch<4, 1, 8, 2, 2>(a, rows, s);
    case 42: return launch<4, 2, 8, 1, 3>(a, rows, s);
    default: return launch<4, 4, 8, 1, 2>(a, rows, s);
  }
}

}  // namespace sp24
