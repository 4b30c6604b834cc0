// Routing tokens to experts: scores of a row of logits, an optional bias for the choice, an optional
// limit to the best groups of experts, the best `top` of what is left and their weights.
//
//   score_i = softmax(l)_i or sigmoid(l_i);   choice c_i = score_i + bias_i, without a bias l_i itself
//   (both scores rise with l);   c_i = -inf where l_i is -inf or NaN: such an expert is taken last, in
//   the order of the indices, and with a -inf its weight is 0.
// Scores that are compared (with a bias, or summed for a group) are formed in 64 bits: among hundreds of
// experts two fp32 scores within a rounding of each other are met every few thousand tokens, and the
// choice would depend on the rounding.
//
// A wave takes a token, lane l the experts l, l + 64, ...
#include "sp24_int4.hpp"

namespace sp24 {
namespace {

constexpr double kNone = -__builtin_inf();

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v = fmax(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
  return v;
}
// The largest value of the wave and the lowest index that has it.
__device__ __forceinline__ void wave_best(double& v, int& i) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const double w = __shfl_xor(v, o);
    const int j = __shfl_xor(i, o);
    if (w > v || (w == v && j < i)) {
      v = w;
      i = j;
    }
  }
}

// NV values a lane: experts <= 64 NV.
template <int NV, bool BF16>
__global__ __launch_bounds__(256) void route_kernel(sp24_router r, int64_t tokens, const void* __restrict__ logits,
                                                    const float* __restrict__ bias, int32_t* __restrict__ ids,
                                                    float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  if (t >= tokens) return;  // whole waves
  const int E = (int)r.experts;
  const bool soft = r.kind == SP24_ROUTE_SOFTMAX;
  double l[NV], score[NV], c[NV];
  double top = kNone;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    l[i] = kNone;
    if (e < E) {
      l[i] = BF16 ? (double)bf16_to_f32(static_cast<const uint16_t*>(logits)[t * E + e])
                  : (double)static_cast<const float*>(logits)[t * E + e];
      l[i] = l[i] > 3.4028234663852886e38 ? 3.4028234663852886e38 : l[i];  // +inf: the largest number
      top = fmax(top, l[i]);  // drops a NaN
    }
  }
  top = wave_max(top);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    // -inf: 0, also where all of them are; NaN stays one
    score[i] = l[i] == kNone ? 0.0 : soft ? exp(l[i] - top) : 1.0 / (1.0 + exp(-l[i]));
    sum += score[i];
  }
  if (soft) {
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < NV; ++i) score[i] = sum == 0.0 ? 0.0 : score[i] / sum;
  }
  bool taken[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    taken[i] = e >= E;
    c[i] = !(l[i] > kNone) ? kNone : bias != nullptr && e < E ? score[i] + (double)bias[e] : l[i];
    if (c[i] != c[i]) c[i] = kNone;  // a bias or a sum that is NaN
  }

  if (r.groups > 1) {
    // a group's value: the sum of its best one or two; the best top_groups groups stay
    const int per = E / (int)r.groups;
    const bool scores = bias == nullptr && r.group_best == 2;
    double value = kNone;  // of group `lane`; groups <= 64
    for (int g = 0; g < r.groups; ++g) {
      double best = kNone, second = kNone;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 64 * i;
        if (e < g * per || e >= (g + 1) * per || c[i] == kNone) continue;
        const double v = scores ? score[i] : c[i];
        second = fmax(second, fmin(best, v));
        best = fmax(best, v);
      }
#pragma unroll
      for (int o = 1; o < 64; o *= 2) {
        const double b2 = __shfl_xor(best, o), s2 = __shfl_xor(second, o);
        second = fmax(fmax(second, s2), fmin(best, b2));
        best = fmax(best, b2);
      }
      if (r.group_best == 2 && second > kNone) best += second;
      if (lane == g) value = best;
    }
    uint64_t keep = 0;
    bool used = lane >= r.groups;
    for (int j = 0; j < r.top_groups; ++j) {
      double v = used ? kNone : value;
      int g = used ? 1 << 20 : lane;
      wave_best(v, g);
      keep |= (uint64_t)1 << g;
      used = used || lane == g;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E) taken[i] = (keep >> (e / per) & 1) == 0;
    }
  }

  // slot j's expert and score end in lane j (top <= 64)
  int id = 0;
  double won = 0.0, at = kNone;
  for (int j = 0; j < r.top; ++j) {
    double v = kNone;
    int e = 1 << 20;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!taken[i] && (e == 1 << 20 || c[i] > v)) {
        v = c[i];
        e = lane + 64 * i;
      }
    wave_best(v, e);
    double sc = 0.0, lv = kNone;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e == lane + 64 * i) {
        taken[i] = true;
        sc = score[i];
        lv = l[i];
      }
    sc = __shfl(sc, e & 63);
    lv = __shfl(lv, e & 63);
    if (lane == j) {
      id = e;
      won = sc;
      at = lv;
    }
  }
  if (r.renormalise) {
    if (soft) {  // relative to the largest that was chosen: none of them underflows
      const double big = wave_max(at);  // drops a NaN
      won = lane < r.top ? (at == kNone ? 0.0 : exp(at - big)) : 0.0;
    }
    const double all = wave_sum(lane < r.top ? won : 0.0);
    won = all == 0.0 ? 0.0 : won / all;
  }
  if (lane < r.top) {
    ids[t * r.top + lane] = id;
    weights[t * r.top + lane] = (float)(won * (double)r.factor);
  }
}

template <int NV>
hipError_t launch(const sp24_router& r, int64_t tokens, const void* logits, const float* bias, int32_t* ids,
                  float* weights, hipStream_t s) {
  const dim3 grid((uint32_t)((tokens + 3) / 4)), block(256);
  if (r.logits_fp32)
    hipLaunchKernelGGL((route_kernel<NV, false>), grid, block, 0, s, r, tokens, logits, bias, ids, weights);
  else
    hipLaunchKernelGGL((route_kernel<NV, true>), grid, block, 0, s, r, tokens, logits, bias, ids, weights);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const sp24_router& r, int64_t tokens, const void* logits, const float* bias, int32_t* ids,
                        float* weights, hipStream_t s) {
  if (r.experts <= 64) return launch<1>(r, tokens, logits, bias, ids, weights, s);
  if (r.experts <= 256) return launch<4>(r, tokens, logits, bias, ids, weights, s);
  return launch<16>(r, tokens, logits, bias, ids, weights, s);
}

}  // namespace sp24
