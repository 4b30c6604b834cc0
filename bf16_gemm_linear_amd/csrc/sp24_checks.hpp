// Argument checks and launch epilogue shared by the C entry points.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>

#include "sp24.h"

namespace sp24 {

constexpr int64_t kMaxDim = (int64_t)1 << 30;

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool overlaps(const void* a, size_t abytes, const void* b, size_t bbytes) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + bbytes && b0 < a0 + abytes;
}

struct Span {
  const void* p;
  size_t bytes;
};

// every output against every input and every other output (NULL spans are skipped)
template <int NI, int NO>
bool any_alias(const Span (&in)[NI], const Span (&out)[NO]) {
  for (int o = 0; o < NO; ++o) {
    if (out[o].p == nullptr || out[o].bytes == 0) continue;
    for (int i = 0; i < NI; ++i)
      if (in[i].p != nullptr && overlaps(out[o].p, out[o].bytes, in[i].p, in[i].bytes)) return true;
    for (int j = o + 1; j < NO; ++j)
      if (out[j].p != nullptr && overlaps(out[o].p, out[o].bytes, out[j].p, out[j].bytes)) return true;
  }
  return false;
}

// Parts of a workspace begin at multiples of 256 bytes.
inline size_t pad(size_t b) { return (b + 255) / 256 * 256; }

inline bool sync_check_enabled() {
  static const bool on = [] {
    const char* v = getenv("SP24_SYNC_CHECK");
    return v != nullptr && v[0] != '\0' && v[0] != '0';
  }();
  return on;
}

inline int finish(hipError_t launch, hipStream_t s) {
  if (launch != hipSuccess) return SP24_ERR_HIP;
  if (sync_check_enabled()) {
    if (hipStreamSynchronize(s) != hipSuccess) return SP24_ERR_HIP;
    if (hipGetLastError() != hipSuccess) return SP24_ERR_HIP;
  }
  return SP24_OK;
}

}  // namespace sp24
