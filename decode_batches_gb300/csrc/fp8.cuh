// 8-bit (e4m3) blocks with an fp32 scale: the quantisation rule shared by every kernel that
// writes such values, and the tensor-core helpers of the 8-bit product.
//
// One block of 128 elements (activations) or 128 x 128 (weights) with largest magnitude `amax`:
//     s = max(amax / 448, 2^-126),   r = fl(1 / s),   q = e4m3(fl(v * r)),   v ~ q * s.
// The scale and the two products are fp32 (each correctly rounded), the last step rounds to
// nearest even; |v * r| <= 448 (1 + 2^-22), which e4m3 rounds to 448, its largest value.  An
// all-zero block has s = 2^-126 and codes 0.  A NaN element keeps the code of NaN; an infinite
// one makes s infinite and the block NaN.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kF8Block = 128;             // elements that share a scale
constexpr float kE4m3Max = 448.0f;
constexpr float kF8ScaleMin = 1.1754943508222875e-38f;  // 2^-126

MOE_DEVICE float f8_scale(float amax) { return fmaxf(__fdiv_rn(amax, kE4m3Max), kF8ScaleMin); }

// e4m3 codes of two values, `lo` in the low byte.
MOE_DEVICE uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, kind::f8f6f4 (e4m3 x e4m3, fp32 accumulate, K = 32).
MOE_DEVICE void mma_f8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4: D fp32 (bits 4-5 = 1), A and B e4m3 (bits 7-9 and 10-12 =
// 0), both K-major, N >> 3 in bits [17,23), M >> 4 in bits [24,29).
MOE_DEVICE uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) { return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24); }

// Wait for this thread's TMEM loads; the registers pass through so that no use moves above it.
MOE_DEVICE void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// Two fp32 lanes in one register pair: acc += v * s, each correctly rounded.
MOE_DEVICE uint64_t pack_f32x2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
MOE_DEVICE void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
MOE_DEVICE void fma_f32x2(uint64_t& acc, uint64_t v, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}

}  // namespace moe
