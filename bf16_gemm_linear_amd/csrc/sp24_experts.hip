// Around the experts' products: the pairs (token, slot) in the order of their experts before them, and
// the weighted sum over a token's slots behind them.
#include "sp24_int4.hpp"
#include "sp24_mx4.hpp"

namespace sp24 {
namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortLoads = 4;  // of a lane's ids in flight

// Workgroup e finds the places of expert e: it counts the ids below e (where its range begins) and lists
// the pairs with id e, in their order, without atomics: a wave takes a run of neighbouring pairs, 64 at a
// time, counts its own in a first pass and, behind the waves before it, places them in a second.  64 experts: 232
// pairs 2.6 us, 14216 pairs 5.8, most of it the two passes' trips to L2.
__global__ __launch_bounds__(kSortThreads) void sort_pairs_kernel(const int32_t* __restrict__ ids, int count,
                                                                  int experts, int* __restrict__ offsets,
                                                                  int* __restrict__ order) {
  __shared__ int sums[kSortWaves][2];
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int run = (count + kSortThreads - 1) / kSortThreads * 64;
  const int from = wave * run, to = min(count, from + run);
  auto load = [&](int i0, int (&id)[kSortLoads]) {
#pragma unroll
    for (int j = 0; j < kSortLoads; ++j) {
      const int i = i0 + 64 * j + lane;
      id[j] = i < to ? ids[i] : -1;
    }
  };
  int below = 0, mine = 0;
  for (int i0 = from; i0 < to; i0 += 64 * kSortLoads) {
    int id[kSortLoads];
    load(i0, id);
#pragma unroll
    for (int j = 0; j < kSortLoads; ++j) {
      mine += __popcll(__ballot(id[j] == e));
      below += __popcll(__ballot(id[j] >= 0 && id[j] < e));
    }
  }
  if (lane == 0) {
    sums[wave][0] = mine;
    sums[wave][1] = below;
  }
  __syncthreads();
  int start = 0, before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    start += sums[w][1];
    before += w < wave ? sums[w][0] : 0;
    all += sums[w][0];
  }
  if (tid == 0) {
    offsets[e] = start;
    if (e == experts - 1) offsets[experts] = start + all;
  }
  int at = start + before;
  for (int i0 = from; i0 < to; i0 += 64 * kSortLoads) {
    int id[kSortLoads];
    load(i0, id);
#pragma unroll
    for (int j = 0; j < kSortLoads; ++j) {
      const uint64_t here = __ballot(id[j] == e);
      if (here >> lane & 1) order[at + __popcll(here & (((uint64_t)1 << lane) - 1))] = i0 + 64 * j + lane;
      at += __popcll(here);
    }
  }
}

// y[t] = sum over slots of weight * part, in the order of the slots; 4 columns a thread (d % 32 == 0).
// HBM: 14216 pairs x 4096 (248 MB) 44 us.
__global__ __launch_bounds__(256) void join_pairs_kernel(const float* __restrict__ part,
                                                         const int32_t* __restrict__ ids,
                                                         const float* __restrict__ weights, int64_t units, int quads,
                                                         int top, int experts, uint16_t* __restrict__ y) {
  constexpr int J = 8;  // slots whose loads are in flight together
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const int64_t t = u / quads;
    const int q = (int)(u - t * quads);
    f32x4 sum{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < top; j0 += J) {
      f32x4 v[J];
      float w[J];
#pragma unroll
      for (int i = 0; i < J; ++i) {
        const int64_t p = t * top + min(j0 + i, top - 1);
        const bool there = j0 + i < top && (uint32_t)ids[p] < (uint32_t)experts;
        v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        w[i] = there ? weights[p] : 0.0f;
        if (there) v[i] = reinterpret_cast<const f32x4*>(part)[p * quads + q];
      }
#pragma unroll
      for (int i = 0; i < J; ++i) sum += w[i] * v[i];
    }
    reinterpret_cast<u32x2*>(y)[u] = u32x2{f32x2_to_bf16x2(sum[0], sum[1]), f32x2_to_bf16x2(sum[2], sum[3])};
  }
}

}  // namespace

hipError_t launch_sort_pairs(const int32_t* ids, int64_t count, int experts, int* offsets, int* order, hipStream_t s) {
  hipLaunchKernelGGL(sort_pairs_kernel, dim3(experts), dim3(kSortThreads), 0, s, ids, (int)count, experts, offsets,
                     order);
  return hipGetLastError();
}

hipError_t launch_join_pairs(const float* part, const int32_t* ids, const float* weights, int64_t tokens, int top,
                             int experts, int d, uint16_t* y, hipStream_t s) {
  const int64_t units = tokens * (d / 4), blocks = (units + 255) / 256;
  hipLaunchKernelGGL(join_pairs_kernel, dim3((uint32_t)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, part, ids,
                     weights, units, d / 4, top, experts, y);
  return hipGetLastError();
}

}  // namespace sp24
