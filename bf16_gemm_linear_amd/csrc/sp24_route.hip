// Routing tokens to experts: scores of a row of logits, an optional bias for the choice, an optional
// limit to the best groups of experts, the best `top` of what is left and their weights.
//
//   score_i = softmax(l)_i or sigmoid(l_i);   choice c_i = score_i + bias_i, without a bias l_i itself
//   (both scores rise with l).   A NaN counts as -inf: c_i = -inf and score 0, so that such an expert is
//   taken last, in the order of the indices, with weight 0, and the others' scores do not know of it.
// Scores that are compared (with a bias, or summed for a group) are formed in 64 bits: among hundreds of
// experts two fp32 scores within a rounding of each other are met every few thousand tokens, and the
// choice would depend on the rounding.  Without them the logits are compared, in fp32, as they are.
//
// A wave takes a token.  The lanes are dealt to the groups, a power of two to each, and a lane holds V
// neighbouring experts of its group, so that a group's value is a reduction over its lanes, all groups at
// once, and the lowest lane that holds a value has the lowest index.  An expert that was taken, or is in no chosen
// group, is NaN, which maxima pass over.  Reductions are register exchanges (sp24_mx4.hpp's).  The weights are
// formed by the first `top` lanes, each from its expert's logit, in 64 bits.
//
// One token takes 2.6 us, a launch and a trip to memory; 8191 tokens x 256 experts in 8 groups with a bias, 8 taken,
// 14.5 a call: some 850 vector instructions a token, 30 of them a pick, not its 1 KB, which alone would take 1.7.
// 4000 x 60, 4 taken: 4.1 a call.
#include "sp24_int4.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

// A logit as it counts: +inf as the largest number, NaN as -inf.
__device__ __forceinline__ float logit(float v) {
  return v != v ? -__builtin_inff() : v > 3.402823466e38f ? 3.402823466e38f : v;
}

// The unsigned numbers whose order is that of a double's upper word or of a float (no NaN: the least; no -0).
__device__ __forceinline__ uint32_t order_key(uint32_t bits, bool number) {
  return number ? bits ^ ((uint32_t)((int32_t)bits >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ uint32_t order_key(float v) { return order_key(__float_as_uint(v), v == v); }
__device__ __forceinline__ uint32_t order_key(double v) {
  return order_key((uint32_t)(__builtin_bit_cast(uint64_t, v) >> 32), v == v);
}

// The value of the lane OFF away (for 4 and 8 one of the aligned group of OFF lanes there).
template <int OFF, class T>
__device__ __forceinline__ void pair_of(T v, T& a, T& b) {
  if constexpr (sizeof(T) == 8) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t l0, l1, h0, h1;
    pair_of<OFF>((uint32_t)u, l0, l1);
    pair_of<OFF>((uint32_t)(u >> 32), h0, h1);
    a = __builtin_bit_cast(T, (uint64_t)h0 << 32 | l0);
    b = __builtin_bit_cast(T, (uint64_t)h1 << 32 | l1);
  } else {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    if constexpr (OFF == 32) {
      const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
      a = __builtin_bit_cast(T, (uint32_t)r[0]);
      b = __builtin_bit_cast(T, (uint32_t)r[1]);
    } else if constexpr (OFF == 16) {
      const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
      a = __builtin_bit_cast(T, (uint32_t)r[0]);
      b = __builtin_bit_cast(T, (uint32_t)r[1]);
    } else {
      constexpr int CTRL = OFF == 1 ? 0xB1 : OFF == 2 ? 0x4E : OFF == 4 ? 0x141 : 0x140;
      a = v;
      b = __builtin_bit_cast(T, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, 0xF, 0xF, true));
    }
  }
}
// The larger, of a number and a NaN the number.  The instructions by name: the compiler's fmax first makes every
// operand a quiet NaN in an instruction of its own, which all NaN here are.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double larger(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

template <int OFF, class T>
__device__ __forceinline__ T step_max(T v) {
  T a, b;
  pair_of<OFF>(v, a, b);
  return larger(a, b);
}
template <class T>
__device__ __forceinline__ T wave_max(T v) {
  return step_max<32>(step_max<16>(step_max<8>(step_max<4>(step_max<2>(step_max<1>(v))))));
}
template <int OFF, class T>
__device__ __forceinline__ T step_sum(T v) {
  T a, b;
  pair_of<OFF>(v, a, b);
  return a + b;
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
  return step_sum<32>(step_sum<16>(step_sum<8>(step_sum<4>(step_sum<2>(step_sum<1>(v))))));
}
// the two largest
template <int OFF, class T>
__device__ __forceinline__ void step_two(T& best, T& second) {
  T a, b, c, d;
  pair_of<OFF>(best, a, b);
  pair_of<OFF>(second, c, d);
  best = larger(a, b);
  second = larger(a < b ? a : b, larger(c, d));
}

// e^x to about 2^-51, x <= 0 (below -745: 0): x = k ln 2 + r, the series of e^r to its
// fourteenth term (|r| <= 0.347: the next is below 2^-57).  All V together: the coefficients are loaded once.
template <int V>
__device__ __forceinline__ void exps_of(double (&x)[V]) {
  constexpr double coefficient[] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0,
                                    1.0 / 5040.0,      1.0 / 720.0,      1.0 / 120.0,     1.0 / 24.0,     1.0 / 6.0,
                                    0.5,               1.0,              1.0};
  double k[V], r[V], p[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    k[i] = rint(x[i] * 1.4426950408889634);
    r[i] = fma(k[i], -0.6931471824645996, x[i]);  // ln 2 as the nearest float (k times it is exact) and the rest
    r[i] = fma(k[i], 1.90465429995776805e-09, r[i]);
    p[i] = 1.0 / 6227020800.0;
  }
#pragma unroll
  for (int c = 0; c < 13; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = fma(p[i], r[i], coefficient[c]);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = x[i] < -745.0 ? 0.0 : __builtin_amdgcn_ldexp(p[i], (int)fmax(k[i], -2000.0));
}
__device__ __forceinline__ double exp_of(double x) {
  double v[1] = {x};
  exps_of(v);
  return v[0];
}
// sigmoid of x, e being e^-|x|
__device__ __forceinline__ double sigmoid(double x, double e) { return (x < 0.0 ? e : 1.0) / (1.0 + e); }

struct Shape {
  int experts, top, groups, per, lanes_log2;  // per: experts of a group; 2^lanes_log2 lanes hold it
};

// T: double where scores are compared, float where logits are.
template <class T, int V, bool BF16>
__global__ __launch_bounds__(256) void route_kernel(sp24_router r, Shape s, int64_t tokens,
                                                    const void* __restrict__ logits, const float* __restrict__ bias,
                                                    int32_t* __restrict__ ids, float* __restrict__ weights) {
  constexpr bool WIDE = sizeof(T) == 8;
  const float none = -__builtin_inff();
  const T gone = __builtin_nanf("");
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  if (t >= tokens) return;  // whole waves
  const bool soft = r.kind == SP24_ROUTE_SOFTMAX;
  const int group = lane >> s.lanes_log2, in = (lane & ((1 << s.lanes_log2) - 1)) * V;
  const int e0 = group * s.per + in;                                    // this lane's experts: e0 .. e0 + held - 1
  const int held = group < s.groups ? max(0, min(V, s.per - in)) : 0;
  const int64_t row = t * s.experts;

  float l[V];
  if (V % 4 == 0 && s.per % 4 == 0) {  // then so are the row and held
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      f32x4 v{none, none, none, none};
      if (i < held) {
        if constexpr (BF16) {
          const u32x2 u = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(logits) + row + e0 + i);
          v = f32x4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xFFFF0000u), __uint_as_float(u[1] << 16),
                    __uint_as_float(u[1] & 0xFFFF0000u)};
        } else {
          v = *reinterpret_cast<const f32x4*>(static_cast<const float*>(logits) + row + e0 + i);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < V) l[i + j] = v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = none;
      if (i < held)
        l[i] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(logits)[row + e0 + i])
                    : static_cast<const float*>(logits)[row + e0 + i];
    }
  }
  float most = none;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    l[i] = logit(l[i]);
    most = larger(most, l[i]);
  }
  if (soft) most = wave_max(most);
  // a row without numbers has no e^(l - most); its scores are 0
  const float from = most == none ? 0.0f : most;

  T c[V];
  double sum = 1.0;  // of e^(l - most), for the softmax
  T best = none, second = none;
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i] == none ? -1000.0 : soft ? (double)l[i] - from : -fabs((double)l[i]);
    exps_of(c);  // 0 for -1000
    if (soft) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += c[i];
      sum = wave_sum(sum);
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = sum == 0.0 ? 0.0 : c[i] / sum;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = sigmoid((double)l[i], c[i]);  // of -inf: 0
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double score = c[i];
      c[i] = bias != nullptr && i < held ? score + (double)bias[e0 + i] : (double)l[i];
      if (!(l[i] > none) || c[i] != c[i]) c[i] = none;  // masked, or a bias that is NaN
      // the group's value is of choices, without a bias of scores
      const double v = bias != nullptr ? c[i] : score;
      if (c[i] != none) {
        second = larger(second, best < v ? best : v);
        best = larger(best, v);
      }
      c[i] = i < held ? c[i] + 0.0 : gone;  // no -0
    }
  } else {
    if (soft && !r.renormalise) {
      double x[V];
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = l[i] == none ? -1000.0 : (double)l[i] - from;
      exps_of(x);
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += x[i];
      sum = wave_sum(sum);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = l[i] > none ? l[i] : none;
      best = larger(best, c[i]);
      c[i] = i < held ? c[i] + 0.0f : gone;  // no -0
    }
  }

  if (s.groups > 1) {
    // over the group's lanes, step by step
    if (s.lanes_log2 > 0) step_two<1>(best, second);
    if (s.lanes_log2 > 1) step_two<2>(best, second);
    if (s.lanes_log2 > 2) step_two<4>(best, second);
    if (s.lanes_log2 > 3) step_two<8>(best, second);
    if (s.lanes_log2 > 4) step_two<16>(best, second);
    T value = best;
    if (WIDE && r.group_best == 2 && second > none) value += second;
    int before = 0;  // groups that come before this lane's
    for (int g = 0; g < s.groups; ++g) {
      T v;
      if constexpr (WIDE) {
        const uint64_t u = __builtin_bit_cast(uint64_t, value);
        const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, g << s.lanes_log2);
        const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), g << s.lanes_log2);
        v = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
      } else {
        v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(value), g << s.lanes_log2));
      }
      before += v > value || (v == value && g < group);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (before >= r.top_groups) c[i] = gone;
  }

  // slot j's expert ends in lane j (top <= 64)
  int id = 0;
  if constexpr (V <= 4) {
    // Few values a lane: sorted once, the best first and of equal ones the lower index, so that a pick looks at
    // every lane's first alone and the winner's move up (8191 x 256, 32 taken: 23.4 us from 28.5; 8 taken 13.9 from
    // 14.6).  As 32-bit words in their order: a double's upper one and, for those equal, its lower one.  Sorting
    // more than four would take longer than the picks.
    int e[V];
    uint32_t key[V], low[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = e0 + i;
#pragma unroll
    for (int n = V - 1; n > 0; --n)
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const bool swap = c[i + 1] > c[i];  // never with one that is gone: those come last or are all
        const T a = c[i], b = c[i + 1];
        const int f = e[i], g = e[i + 1];
        c[i] = swap ? b : a;
        c[i + 1] = swap ? a : b;
        e[i] = swap ? g : f;
        e[i + 1] = swap ? f : g;
      }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = order_key(c[i]);
      if constexpr (WIDE) {
        const uint32_t u = (uint32_t)__builtin_bit_cast(uint64_t, c[i]);
        low[i] = key[i] >> 31 ? u : ~u;
      }
    }
    for (int j = 0; j < s.top; ++j) {
      const uint32_t most_key = fold_wave(key[0], bits_max);
      uint64_t first = __ballot(key[0] == most_key);
      if (WIDE && (first & (first - 1)) != 0) {
        asm volatile("");  // a branch, not both sides
        const uint32_t most_low = fold_wave(key[0] == most_key ? low[0] : 0u, bits_max);
        first &= __ballot(low[0] == most_low);
      }
      const int winner = __ffsll((unsigned long long)first) - 1;
      const int taken = __builtin_amdgcn_readlane(e[0], winner);
      const bool here = lane == winner;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i + 1 < V) {
          const uint32_t k = key[i], next = key[i + 1];
          key[i] = here ? next : k;
          if constexpr (WIDE) {
            const uint32_t l0 = low[i], l1 = low[i + 1];
            low[i] = here ? l1 : l0;
          }
          const int f = e[i], g = e[i + 1];
          e[i] = here ? g : f;
        } else {
          key[i] = here ? 0u : key[i];  // gone
        }
      }
      if (lane == j) id = taken;
    }
  } else {
    for (int j = 0; j < s.top; ++j) {
      T v = c[0];
#pragma unroll
      for (int i = 1; i < V; ++i) v = larger(v, c[i]);
      int at = 0;  // the first of this lane's with that value
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (c[i] == v) at = i;
      // 32 bits of each lane's best are compared; all of them only where those are equal
      const uint32_t key = order_key(v);
      uint32_t most_key = fold_wave(key, bits_max);
      uint64_t first = __ballot(key == most_key);
      if (WIDE && (first & (first - 1)) != 0) {
        asm volatile("");  // a branch, not both sides
        const T all = wave_max(key == most_key ? v : gone);
        first = __ballot(v == all);
      }
      const int winner = __ffsll((unsigned long long)first) - 1;
      const int e = __builtin_amdgcn_readlane(e0 + at, winner);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane == winner && i == at) c[i] = gone;
      if (lane == j) id = e;
    }
  }

  double won = 0.0;
  float at = none;
  const bool mine = lane < s.top;
  if (mine)
    at = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(logits)[row + id])
              : static_cast<const float*>(logits)[row + id];
  at = logit(at);
  if (soft) {
    // renormalised: relative to the largest that was chosen, so that none of them underflows
    const float big = r.renormalise ? wave_max(at) : from;
    won = mine && at != none ? exp_of((double)at - (big == none ? 0.0f : big)) : 0.0;
    if (!r.renormalise && sum != 0.0) won /= sum;
  } else {
    won = mine && at != none ? sigmoid((double)at, exp_of(-fabs((double)at))) : 0.0;
  }
  if (r.renormalise) {
    const double all = wave_sum(won);
    won = all == 0.0 ? 0.0 : won / all;
  }
  if (mine) {
    ids[t * s.top + lane] = id;
    weights[t * s.top + lane] = (float)(won * (double)r.factor);
  }
}

template <class T, int V>
hipError_t launch(const sp24_router& r, const Shape& p, int64_t tokens, const void* logits, const float* bias,
                  int32_t* ids, float* weights, hipStream_t s) {
  const dim3 grid((uint32_t)((tokens + 3) / 4)), block(256);
  if (r.logits_fp32)
    hipLaunchKernelGGL((route_kernel<T, V, false>), grid, block, 0, s, r, p, tokens, logits, bias, ids, weights);
  else
    hipLaunchKernelGGL((route_kernel<T, V, true>), grid, block, 0, s, r, p, tokens, logits, bias, ids, weights);
  return hipGetLastError();
}

template <class T>
hipError_t by_size(const sp24_router& r, const Shape& p, int64_t tokens, const void* logits, const float* bias,
                   int32_t* ids, float* weights, hipStream_t s) {
  const int v = (p.per + (1 << p.lanes_log2) - 1) >> p.lanes_log2;  // at most 32: 31 experts a lane of 33 groups
  if (v <= 1) return launch<T, 1>(r, p, tokens, logits, bias, ids, weights, s);
  if (v <= 2) return launch<T, 2>(r, p, tokens, logits, bias, ids, weights, s);
  if (v <= 4) return launch<T, 4>(r, p, tokens, logits, bias, ids, weights, s);
  if (v <= 8) return launch<T, 8>(r, p, tokens, logits, bias, ids, weights, s);
  if (v <= 16) return launch<T, 16>(r, p, tokens, logits, bias, ids, weights, s);
  return launch<T, 32>(r, p, tokens, logits, bias, ids, weights, s);
}

}  // namespace

hipError_t launch_route(const sp24_router& r, int64_t tokens, const void* logits, const float* bias, int32_t* ids,
                        float* weights, hipStream_t s) {
  Shape p{(int)r.experts, (int)r.top, (int)r.groups, (int)(r.experts / r.groups), 6};
  while (p.groups << p.lanes_log2 > 64) --p.lanes_log2;
  const bool wide = bias != nullptr || (r.groups > 1 && r.group_best == 2);
  return wide ? by_size<double>(r, p, tokens, logits, bias, ids, weights, s)
              : by_size<float>(r, p, tokens, logits, bias, ids, weights, s);
}

}  // namespace sp24
