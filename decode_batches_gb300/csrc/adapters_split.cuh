// Device helpers that both adapter kernels use.
#pragma once

#include "elems.cuh"

namespace moe {

// Asks L2 for `bytes` from p (16-byte aligned, a multiple of 16).
MOE_DEVICE void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// counts[key] += 1 for every lane with a key >= 0, and what was there before this lane's: a run of one key (a prompt's
// rows) with one addition, else a lane's each, whose few collisions take less time than to find them (10 us of 22 at
// 30000 rows).
MOE_DEVICE int count_key(int* counts, int key, int lane) {
  if (__all_sync(0xffffffffu, key == __shfl_sync(0xffffffffu, key, 0)) && key >= 0) {
    int at = 0;
    if (lane == 0) at = atomicAdd(&counts[key], 32);
    return __shfl_sync(0xffffffffu, at, 0) + lane;
  }
  return key >= 0 ? atomicAdd(&counts[key], 1) : 0;
}

// Eight elements of a row of x from column c (zeros past K), at any alignment.
MOE_DEVICE uint4 load_x(const uint16_t* row, int c, int K) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = c + 2 * i < K ? row[c + 2 * i] : 0u, hi = c + 2 * i + 1 < K ? row[c + 2 * i + 1] : 0u;
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16-bit terms that hold u: in bf16 three, whose 24 bits are all that an fp32 sum has (with two, an fp32 result of 2048 x 4096
// and rank 16 was 2.5e-6 off the formula where fp32 products are 1.5e-7 off); in fp16 two, 22 bits.
template <bool kFp16>
constexpr int kAdapterTerms = kFp16 ? 2 : 3;

// Ranks c .. c + 7 of a row's sums as the terms of u = scale * v (0 behind the slot's rank, where an infinite x
// makes NaN of the padding); R / 8 neighbouring lanes hold a row.  Returns what the terms were divided by: 1 in bf16;
// in fp16 the power of two that brings the row's largest u to [2^14, 2^15): neither term leaves the type's range, and a u
// keeps its 22 bits down to 2^-17 of the largest (with the largest in [1, 2), one 2^-10 below it had 14 left).
// (1 for a row that is zero, infinite or NaN.)
template <int R, bool kFp16>
MOE_DEVICE float adapter_split(float (&v)[8], int c, int rank, float scale, uint4 (&term)[kAdapterTerms<kFp16>]) {
  float mul = 1.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = c + e < rank ? v[e] * scale : 0.0f;
  if (kFp16) {
    float big = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(v[e]));
#pragma unroll
    for (int o = 1; o < R / 8; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    const int ex = static_cast<int>(__float_as_uint(big) >> 23) - 127;  // big in [2^ex, 2^(ex + 1))
    const int e2 = ex == -127 || ex == 128 ? 0 : max(-126, ex - 14);
    mul = __uint_as_float(static_cast<uint32_t>(e2 + 127) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= down;
  }
#pragma unroll
  for (int t = 0; t < kAdapterTerms<kFp16>; ++t) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      float h0, h1;
      if (kFp16) {
        w[e / 2] = pack_f16x2(v[e], v[e + 1]);
        h0 = f16_bits_to_f32(w[e / 2] & 0xffffu), h1 = f16_bits_to_f32(w[e / 2] >> 16);
      } else {
        w[e / 2] = cvt_bf16x2(v[e], v[e + 1]);
        h0 = bf16_bits_to_f32(w[e / 2] & 0xffffu), h1 = bf16_bits_to_f32(w[e / 2] >> 16);
      }
      // (an infinity has no rest)
      v[e] = isfinite(h0) ? v[e] - h0 : 0.0f, v[e + 1] = isfinite(h1) ? v[e + 1] - h1 : 0.0f;
    }
    term[t] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return mul;
}

}  // namespace moe
