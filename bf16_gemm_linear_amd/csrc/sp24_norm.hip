// RMS norm with the residual's addition, its output in bf16, in 8 bits with scales or in
// MXFP4: per row, t = x + residual (fp32, unrounded; bf16_rne(t) is the new residual),
// v = t rstd w with rstd = 1 / sqrt(mean(t^2) + eps).
//
// Memory-bound: 2 bytes read a value (6 moved with a residual) and 1 written (E4M3, INT8).
// 8191 x 8192 with a residual takes 78 to 81 us to E4M3 with a scale per row, 81 with one per group
// of 128, 74 to 76 to MXFP4 and 91 to bf16, 5.8 TB/s (a large copy: 5.1); the outputs' non-temporal hint is worth
// a quarter of it where the inputs come from the last-level cache (68 us, 89 without).  Few rows
// are bound by a thread's chain of instructions: reductions over lanes go by register exchanges
// (through LDS: 1 x 4096 with a residual to E4M3 3.1 us, per group 4.1; now 2.7 and 3.0, 1.7 any
// launch's).
// One pass: a row stays in registers as fp32 from the loads to the codes, T threads a row
// with NV vectors of 8 values each.  The codes do not wait for rstd: with u = t w, a scale
// is s = max|u| rstd / top, so v / s = u (top / max|u|), and one reduction over the row
// gives sum t^2 and max|u| together (for groups, the maxima are taken by shuffles at the
// same time).  Where a maximum of |u| has left fp32's range, or comes so near its lower end
// that values would lose bits (very large or small weights), v itself may be in range: such a
// row takes the maxima of |t rstd w| in a second reduction.  For that t stays in the registers,
// and t w is formed twice: up to 4% of a call (7% with groups of several waves: 8191 x 8192 per
// group of 1024 50 us from 46.5), 10% past 32768 values, where the weight is loaded again (1024 x
// 65536 to E4M3 49 us from 44).  Sums are fp32 in a fixed order.
#include "sp24_fp8.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

// The codes' divisor for values u with largest magnitude amax and scale a / top, a = amax
// rstd: u (top / amax), the factor kept as hi + lo so that the quotient carries one
// rounding; maxima below 2^-60 are scaled up by 2^80 first (exact), so that the factor
// stays finite.  a = 0: scale 1, codes 0.  a Inf or NaN: scale NaN, codes 0.
struct NormDiv {
  float hi, lo, up;
  bool on;
};

template <int KIND>
__device__ __forceinline__ float norm_scale(uint32_t key, float rstd, NormDiv& d) {
  constexpr float top = KIND == SP24_NORM_INT8_ROWS ? 127.0f : 448.0f;
  const float amax = __uint_as_float(key), a = amax * rstd;
  d.on = a > 0.0f && a < __builtin_inff();
  d.up = amax < 0x1p-60f ? 0x1p80f : 1.0f;
  const float b = amax * d.up;
  d.hi = top / b;
  d.lo = __builtin_fmaf(-d.hi, b, top) * (d.hi * (1.0f / top));  // the residual times 1 / b
  const float q = a * (1.0f / top), s = __builtin_fmaf(__builtin_fmaf(-q, top, a), 1.0f / top, q);  // a / top
  return a == 0.0f ? 1.0f : d.on ? s : __uint_as_float(0x7FC00000u);
}

template <int KIND>
__device__ __forceinline__ u32x2 norm_codes8(const float* u, const NormDiv& d) {
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = u[e] * d.up;
    q[e] = d.on ? __builtin_fmaf(t, d.hi, t * d.lo) : 0.0f;
  }
  if constexpr (KIND == SP24_NORM_INT8_ROWS) {
    return u32x2{f32_to_i8(q[0]) | (f32_to_i8(q[1]) << 8) | (f32_to_i8(q[2]) << 16) | (f32_to_i8(q[3]) << 24),
                 f32_to_i8(q[4]) | (f32_to_i8(q[5]) << 8) | (f32_to_i8(q[6]) << 16) | (f32_to_i8(q[7]) << 24)};
  } else {
    return u32x2{f32x2_to_e4m3(q[0], q[1]) | (f32x2_to_e4m3(q[2], q[3]) << 16),
                 f32x2_to_e4m3(q[4], q[5]) | (f32x2_to_e4m3(q[6], q[7]) << 16)};
  }
}

// Value e of a vector of 8 bf16.
__device__ __forceinline__ float bf16_of(const u32x4& d, int e) {
  return __uint_as_float((e & 1) ? d[e / 2] & 0xFFFF0000u : d[e / 2] << 16);
}

// Whether products u = t w with this largest magnitude (bits) may not stand for v: it is Inf or
// NaN, or below 2^-100, where a product under 2^-126 (fewer bits) still counts beside it.
__device__ __forceinline__ bool out_of_range(uint32_t key) { return key >= 0x7F800000u || key < 0x0D800000u; }

// T threads a row (64: one wave, four rows a workgroup; 128: two rows), NV vectors of 8 values a thread.
// Groups (SP24_NORM_FP8_GROUPS): segments of `seg` lanes, seg a power of two dividing the
// group's vectors; where a group is more than one segment its maximum is collected in LDS
// (integer maxima: the order does not matter).
template <int KIND, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rmsnorm_kernel(
    const uint16_t* __restrict__ x, const uint16_t* residual, uint16_t* residual_out,
    const uint16_t* __restrict__ w, int64_t m, int k, float eps, int group, int seg, int ng,
    uint32_t per_group, void* __restrict__ out, void* __restrict__ scales) {
  constexpr int RPB = T < 256 ? 256 / T : 1, NW = T / 64;
  constexpr bool GROUPS = KIND == SP24_NORM_FP8_GROUPS;
  constexpr bool ROWS = KIND == SP24_NORM_FP8_ROWS || KIND == SP24_NORM_INT8_ROWS;
  __shared__ float sh_sum[RPB * NW];
  __shared__ uint32_t sh_max[RPB * NW], sh_max2[RPB * NW];
  extern __shared__ uint32_t gmax[];  // [RPB][groups], only where a group is more than a segment

  const int tl = threadIdx.x % T, rl = threadIdx.x / T, lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * RPB + rl;
  const int nv = row < m ? k / 8 : 0;
  const size_t base = (size_t)row * (k / 8);
  const int vpg = GROUPS ? group / 8 : 1;
  // vector i's group: i / vpg by the factor ceil(2^31 / vpg), exact for i and vpg to 2^13
  auto group_of = [&](int i) { return (int)__umulhi(2u * (uint32_t)i, per_group); };
  const bool in_lds = GROUPS && vpg != seg;
  if (in_lds) {
    for (int i = threadIdx.x; i < RPB * ng; i += (T < 256 ? 256 : T)) gmax[i] = 0;
    __syncthreads();
  }

  // vectors are loaded B at a time: all of a long row's at once would not fit in the registers
  // beside u (1024 x 65536 to E4M3: 134 us, in pairs 43, with the weight loaded again 49)
  constexpr int B = NV > 4 ? 2 : NV;
  constexpr bool KEEP_W = NV <= 4;  // the weight for the output (longer rows load it again, a vector ahead)
  u32x4 wd[KEEP_W ? NV : B];
  float u[NV][8], ss = 0.0f;  // u: t, until the output
  uint32_t key = 0, gkey[NV];
  bool off = false;  // groups: a segment's maximum is out of range

  // a group's maximum from its lanes' (in LDS where a group is more than a segment)
  auto group_max = [&](uint32_t mk) {
    if (seg > 1) mk = fold_lanes<1>(mk, bits_max);
    if (seg > 2) mk = fold_lanes<2>(mk, bits_max);
    if (seg > 4) mk = fold_lanes<4>(mk, bits_max);
    if (seg > 8) mk = fold_lanes<8>(mk, bits_max);
    if (seg > 16) mk = fold_lanes<16>(mk, bits_max);
    if (seg > 32) mk = fold_lanes<32>(mk, bits_max);
    return mk;
  };
  auto collect = [&](uint32_t mk, int i) {
    if (in_lds && i < nv && lane % seg == 0) atomicMax(&gmax[rl * ng + group_of(i)], mk);
  };
#pragma unroll
  for (int j0 = 0; j0 < NV; j0 += B) {
    u32x4 xd[B], rd[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int i = tl + (j0 + b) * T;
      xd[b] = rd[b] = wd[b] = u32x4{0u, 0u, 0u, 0u};
      if (i < nv) {
        xd[b] = reinterpret_cast<const u32x4*>(x)[base + i];
        if (residual != nullptr) rd[b] = reinterpret_cast<const u32x4*>(residual)[base + i];
        wd[b] = reinterpret_cast<const u32x4*>(w)[i];
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int j = j0 + b, i = tl + j * T;
      uint32_t mk = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float t = bf16_of(xd[b], e);
        if (residual != nullptr) t += bf16_of(rd[b], e);
        ss = __builtin_fmaf(t, t, ss);
        u[j][e] = t;
      }
      if (residual != nullptr && i < nv) {
        const u32x4 o{f32x2_to_bf16x2(u[j][0], u[j][1]), f32x2_to_bf16x2(u[j][2], u[j][3]),
                      f32x2_to_bf16x2(u[j][4], u[j][5]), f32x2_to_bf16x2(u[j][6], u[j][7])};
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(residual_out) + base + i);
      }
      if constexpr (ROWS || GROUPS) {
#pragma unroll
        for (int e = 0; e < 8; ++e) mk = max(mk, __float_as_uint(u[j][e] * bf16_of(wd[b], e)) & 0x7FFFFFFFu);
        key = max(key, mk);
      }
      if constexpr (GROUPS) {
        gkey[j] = group_max(mk);
        off = off || (i < nv && out_of_range(gkey[j]));
        collect(gkey[j], i);
      }
    }
    if constexpr (B < NV) {  // finish this batch: its maximum now, not at the end
      asm volatile("" : "+v"(key), "+v"(ss));
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  ss = __uint_as_float(fold_wave(__float_as_uint(ss), bits_sum));
  if constexpr (ROWS) key = fold_wave(key, bits_max);
  auto weight = [&](int j) {
    if constexpr (KEEP_W) {
      return wd[j];
    } else {
      const int i = tl + j * T;
      return i < nv ? reinterpret_cast<const u32x4*>(w)[i] : u32x4{0u, 0u, 0u, 0u};
    }
  };
  if constexpr (GROUPS) {
    if (__any(off)) {
      // groups of true zeros (channels without a signal) are in range, or they would cost their
      // rows a second reduction, 10% of 8191 x 8192; zeros of values that are not are out of it
      off = false;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (tl + j * T >= nv) continue;
        if (gkey[j] != 0) {
          off = off || out_of_range(gkey[j]);
        } else {
          const u32x4 wj = weight(j);
#pragma unroll
          for (int e = 0; e < 8; ++e) off = off || (u[j][e] != 0.0f && bf16_of(wj, e) != 0.0f);
        }
      }
    }
    key = __any(off) ? 1u : 0u;
  }
  if constexpr (NW > 1) {
    if (lane == 0) {
      sh_sum[threadIdx.x / 64] = ss;
      sh_max[threadIdx.x / 64] = key;
    }
    __syncthreads();
    ss = 0.0f;
    key = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      ss += sh_sum[rl * NW + i];
      key = max(key, sh_max[rl * NW + i]);
    }
  } else if (in_lds) {
    if (lane == 0) sh_max[threadIdx.x / 64] = key;
    __syncthreads();
  }
  const float rstd = 1.0f / __builtin_sqrtf(ss / (float)k + eps);

  bool again = false;  // u is t rstd in this row, and its maxima are those of |t rstd w|
  if constexpr (ROWS || GROUPS) {
    auto bad = [&](uint32_t row_key) { return GROUPS ? row_key != 0 : out_of_range(row_key); };
    again = nv > 0 && bad(key);
    // barriers are the workgroup's: all its rows come along, those in range keep what they have
    bool any_again = again;
    if constexpr (RPB > 1) {
      if (NW > 1 || in_lds) {
#pragma unroll
        for (int r = 0; r < RPB; ++r) {
          uint32_t rk = 0;
#pragma unroll
          for (int i = 0; i < NW; ++i) rk = max(rk, sh_max[r * NW + i]);
          any_again = any_again || ((int64_t)blockIdx.x * RPB + r < m && bad(rk));
        }
      }
    }
    auto largest = [&](int j) {
      const u32x4 wj = weight(j);
      uint32_t mk = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) mk = max(mk, __float_as_uint(u[j][e] * bf16_of(wj, e)) & 0x7FFFFFFFu);
      return mk;
    };
    if (any_again) {
      if (again) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) u[j][e] *= rstd;
      }
      if constexpr (ROWS) {
        uint32_t mk = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) mk = max(mk, largest(j));
        mk = fold_wave(mk, bits_max);
        if constexpr (NW > 1) {
          if (lane == 0) sh_max2[threadIdx.x / 64] = mk;
          __syncthreads();
          mk = 0;
#pragma unroll
          for (int i = 0; i < NW; ++i) mk = max(mk, sh_max2[rl * NW + i]);
        }
        if (again) key = mk;
      } else {
        if (in_lds) {
          if (again)
            for (int i = tl; i < ng; i += T) gmax[rl * ng + i] = 0;
          __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const uint32_t mk = group_max(largest(j));
          if (again) {
            gkey[j] = mk;
            collect(mk, tl + j * T);
          }
        }
        if (in_lds) __syncthreads();
      }
    }
  }

  const float left = again ? 1.0f : rstd;  // what the 8-bit forms' scales still have to take
  NormDiv d{0.0f, 0.0f, 1.0f, false};
  if constexpr (ROWS) {
    const float s = norm_scale<KIND>(key, left, d);
    if (tl == 0 && nv > 0) static_cast<float*>(scales)[row] = s;
  }
  u32x4 wnext = weight(0);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tl + j * T;
    const u32x4 wj = wnext;
    if (j + 1 < NV) wnext = weight(j + 1);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[j][e] = (ROWS || GROUPS ? u[j][e] : u[j][e] * rstd) * bf16_of(wj, e);
    if constexpr (KIND == SP24_NORM_BF16) {
      if (i < nv) {
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = f32x2_to_bf16x2(u[j][2 * e], u[j][2 * e + 1]);
        __builtin_nontemporal_store(o, static_cast<u32x4*>(out) + base + i);
      }
    } else if constexpr (KIND == SP24_NORM_MXFP4) {
      uint32_t mk = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) mk = max(mk, __float_as_uint(u[j][e]) & 0x7FFFFFFFu);
      const uint32_t byte = mx4_block_byte<23>(mk);  // k % 128 == 0: the 16 lanes of a word are all in the row
      const uint32_t word = mx4_word_of_blocks(byte, lane);
      if (i < nv) {
        __builtin_nontemporal_store(mx4_codes8(u[j], byte), static_cast<uint32_t*>(out) + base + i);
        if ((lane & 15) == 0) static_cast<uint32_t*>(scales)[mx4_scale_word(row, i / 16, m, k)] = word;
      }
    } else {
      if (i < nv) {
        if constexpr (GROUPS) {
          const int g = group_of(i);
          const float s = norm_scale<KIND>(in_lds ? gmax[rl * ng + g] : gkey[j], left, d);
          if (i == g * vpg) static_cast<float*>(scales)[(size_t)row * ng + g] = s;
        }
        __builtin_nontemporal_store(norm_codes8<KIND>(u[j], d), static_cast<u32x2*>(out) + base + i);
      }
    }
    if constexpr (B < NV) __builtin_amdgcn_sched_barrier(0);
  }
}

template <int KIND, int T, int NV>
hipError_t launch_norm_tn(const NormArgs& a, hipStream_t s) {
  constexpr int RPB = T < 256 ? 256 / T : 1;
  int seg = 1;
  size_t lds = 0;
  const uint64_t vpg = (uint64_t)a.group / 8;  // (any k % 8 == 0: one group a row but for SP24_NORM_FP8_GROUPS)
  if (KIND == SP24_NORM_FP8_GROUPS) {
    while (seg < 64 && vpg % (2 * seg) == 0) seg *= 2;
    if (vpg != seg) lds = (size_t)RPB * (a.k / a.group) * 4;
  }
  hipLaunchKernelGGL((rmsnorm_kernel<KIND, T, NV>), dim3((uint32_t)((a.m + RPB - 1) / RPB)),
                     dim3(T < 256 ? 256 : T), lds, s, a.x, a.residual, a.residual_out, a.weight, a.m, (int)a.k,
                     a.eps, (int)a.group, seg, (int)(a.k / a.group),
                     (uint32_t)((((uint64_t)1 << 31) + vpg - 1) / vpg), a.out, a.scales);
  return hipGetLastError();
}

// Threads a row: one vector a thread for short and few rows (to 4096 values, 2^21 in all), where
// the chain of a thread is the time (E4M3, no residual, us: 16 x 2048 on 256 x 1 and 64 x 4 2.7 and
// 3.5, 256 x 4096 on 512 x 1 and 256 x 2 3.0 and 3.2; with more rows it turns round, 1000 x 4096 4.9
// and 4.5, 8191 x 4096 25.0 and 20.4).  Else a wave to 2048 values, then one workgroup with two
// vectors a thread (8191 x 8192 E4M3 per group of 128 and residual on 512 x 2 81, on 1024 x 1 84;
// 16 rows of 8192 3.3 and 3.4), four to 32768 (2048 x 20480 36, on 1024 x 8 52; the lanes past the
// row idle) and eight beyond.
template <int KIND>
hipError_t launch_norm_kind(const NormArgs& a, hipStream_t s) {
  const int64_t nv = a.k / 8;
  if (nv <= 64) return launch_norm_tn<KIND, 64, 1>(a, s);
  if (nv <= 512 && a.m * a.k <= 1 << 21) {
    if (nv <= 128) return launch_norm_tn<KIND, 128, 1>(a, s);
    if (nv <= 256) return launch_norm_tn<KIND, 256, 1>(a, s);
    return launch_norm_tn<KIND, 512, 1>(a, s);
  }
  if (nv <= 256) return launch_norm_tn<KIND, 64, 4>(a, s);
  if (nv <= 512) return launch_norm_tn<KIND, 256, 2>(a, s);
  if (nv <= 1024) return launch_norm_tn<KIND, 512, 2>(a, s);
  if (nv <= 2048) return launch_norm_tn<KIND, 1024, 2>(a, s);
  if (nv <= 4096) return launch_norm_tn<KIND, 1024, 4>(a, s);
  return launch_norm_tn<KIND, 1024, 8>(a, s);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t s) {
  switch (a.kind) {
    case SP24_NORM_BF16: return launch_norm_kind<SP24_NORM_BF16>(a, s);
    case SP24_NORM_FP8_ROWS: return launch_norm_kind<SP24_NORM_FP8_ROWS>(a, s);
    case SP24_NORM_INT8_ROWS: return launch_norm_kind<SP24_NORM_INT8_ROWS>(a, s);
    case SP24_NORM_FP8_GROUPS: return launch_norm_kind<SP24_NORM_FP8_GROUPS>(a, s);
    default: return launch_norm_kind<SP24_NORM_MXFP4>(a, s);
  }
}

}  // namespace sp24
