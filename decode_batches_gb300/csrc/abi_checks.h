// Host-side helpers of the C entry points: argument checks and error messages.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cstdio>

#include "kernels.h"

namespace moe {

inline moe_status bad(moe_status s, const char* msg) { return fail_message(s, msg); }

inline moe_status cuda_fail(const char* what, cudaError_t e) {
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", what, cudaGetErrorString(e));
  cudaGetLastError();  // reported here: a later check of the caller's own launches does not find it again
  return fail_message(MOE_ERR_CUDA, buf);
}
#define LIN_TRY(expr)                                         \
  do {                                                        \
    const cudaError_t _e = (expr);                            \
    if (_e != cudaSuccess) return moe::cuda_fail(#expr, _e);  \
  } while (0)

inline bool known(moe_dtype t) { return t == MOE_BF16 || t == MOE_FP16 || t == MOE_FP32; }
inline size_t elem_bytes(moe_dtype t) { return t == MOE_FP32 ? 4 : 2; }
inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// Rows of `ld` elements that start at p are all 16-byte aligned (one row: its start alone counts).
inline bool rows_aligned16(const void* p, int64_t ld, moe_dtype t, int64_t rows) {
  return aligned(p, 16) && (rows <= 1 || ld * static_cast<int64_t>(elem_bytes(t)) % 16 == 0);
}

inline int current_device() {
  int dev = 0;
  cudaGetDevice(&dev);
  return dev;
}
inline int current_sms() {
  int n = 0;
  const int dev = current_device();
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

}  // namespace moe
