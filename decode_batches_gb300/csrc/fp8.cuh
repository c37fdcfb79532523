// 8-bit (e4m3) blocks with an fp32 scale: the quantisation rule shared by every kernel that
// writes such values, and the tensor-core helpers of the 8-bit product.
//
// One block of 128 elements (activations) or 128 x 128 (weights) with largest magnitude `amax`:
//     s = max(fl(amax * fl(1 / 448)), 2^-126),   r = fl(1 / s),   q = e4m3(fl(v * r)),   v ~ q * s.
// fl is one correctly rounded fp32 operation; the last step rounds to nearest even; |v * r| <=
// 448 (1 + 2^-22), which e4m3 rounds to 448, its largest value.  An all-zero block has s = 2^-126 and codes 0.
// A NaN element keeps the code of NaN; an infinite one makes s infinite and the block NaN.
#pragma once

#include "common.cuh"

#include <cstring>

namespace moe {

constexpr int kF8Block = 128;             // elements that share a scale
constexpr float kE4m3Max = 448.0f;
constexpr float kF8ScaleMin = 1.1754943508222875e-38f;  // 2^-126

MOE_DEVICE float f8_scale(float amax) { return fmaxf(__fmul_rn(amax, 1.0f / kE4m3Max), kF8ScaleMin); }

// e4m3 codes of two values, `lo` in the low byte.
MOE_DEVICE uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}

// 16 consecutive elements as loaded: 16-byte loads where the address and the row's length allow, else
// element by element (zero beyond `n`).
template <typename T>
struct Raw16 {
  static constexpr int kVec = sizeof(T);
  uint4 v[kVec];
  MOE_DEVICE void load(const T* p, int n, bool vec) {
    if (vec && n >= 16) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
      T e[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) e[i] = i < n ? p[i] : T(0.f);
      memcpy(v, e, sizeof v);
    }
  }
  MOE_DEVICE void get(float (&o)[16]) const;
};
template <>
MOE_DEVICE void Raw16<__nv_bfloat16>::get(float (&o)[16]) const {
  float h[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    bf16x8_to_f32(v[i], h);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[8 * i + j] = h[j];
  }
}
template <>
MOE_DEVICE void Raw16<__half>::get(float (&o)[16]) const {
  float h[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f16x8_to_f32(v[i], h);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[8 * i + j] = h[j];
  }
}
template <>
MOE_DEVICE void Raw16<float>::get(float (&o)[16]) const { memcpy(o, v, sizeof o); }

// Rows x [rows][K] in blocks of 128 by the warps first, first + step, ...: a warp takes eight blocks of
// a row at a time and requests its next eight before it works on them.  Eight lanes hold a block
// in registers (16 elements a lane), take its largest magnitude with three shuffles and write 128
// contiguous bytes of codes and the scale.  nb = ceil(K / 128); vec: the rows are 16-byte aligned.
// 8192 x 4096 bf16: 15.4 us in a graph over three inputs (16.0 without the request ahead), 101 MB, bound
// by memory (under ncu, caches cold, 15.5 us with DRAM at 58% of its peak: part of the codes stays in L2).
template <typename T>
MOE_DEVICE void quant_rows_part(const T* __restrict__ x, int64_t ldx, int rows, int K, int nb, bool vec,
                                uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ s, int64_t lds, uint32_t first,
                                uint32_t step) {
  const uint32_t chunks = (nb + 7) / 8;  // of a row
  const int lane = threadIdx.x & 7, part = (threadIdx.x >> 3) & 3;
  const uint32_t step_row = step / chunks, step_chunk = step % chunks;
  uint32_t row = first / chunks, chunk = first % chunks;
  Raw16<T> raw[2];
  auto request = [&]() {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k0 = (8 * chunk + 4 * u + part) * kF8Block + 16 * lane;
      raw[u].load(x + row * ldx + k0, K - k0, vec);
    }
  };
  if (row < static_cast<uint32_t>(rows)) request();
  while (row < static_cast<uint32_t>(rows)) {
    const Raw16<T> now[2] = {raw[0], raw[1]};
    const uint32_t row_now = row, chunk_now = chunk;
    row += step_row;
    chunk += step_chunk;
    if (chunk >= chunks) chunk -= chunks, ++row;
    if (row < static_cast<uint32_t>(rows)) request();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int b = 8 * chunk_now + 4 * u + part;
      float v[16], amax = 0.f;
      now[u].get(v);
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(v[j]));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float sc = f8_scale(amax);
      const float r = __frcp_rn(sc);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = f32x2_to_e4m3x2(v[4 * j] * r, v[4 * j + 1] * r) | (f32x2_to_e4m3x2(v[4 * j + 2] * r, v[4 * j + 3] * r) << 16);
      if (b < nb) {  // columns K .. 128 nb get the code of zero
        *reinterpret_cast<uint4*>(q + row_now * ldq + b * kF8Block + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
        if (lane == 0) s[row_now * lds + b] = sc;
      }
    }
  }
}

// The conversion of x that a routing launch performs on the side: fp16 copy (4-bit experts) or 8-bit
// blocks (8-bit experts), by blocks `block` of `blocks`.
MOE_DEVICE void convert_x8(const XConv& c, int block, int blocks) {
  const uint32_t per = blockDim.x >> 5;
  quant_rows_part(reinterpret_cast<const __nv_bfloat16*>(c.x), c.K, c.rows, c.K, (c.K + kF8Block - 1) / kF8Block, true, c.xq,
                  c.ldq, c.xs, c.lds, block * per + (threadIdx.x >> 5), blocks * per);
}
MOE_DEVICE void convert_x(const XConv& c, uint32_t* err) {
  if (c.xq)
    convert_x8(c, static_cast<int>((blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x),
               static_cast<int>(gridDim.x * gridDim.y * gridDim.z));
  else
    convert_x16(c, err);
}

// One K block of 128: D[tmem] = A[smem desc] * B[smem desc]^T, kind::f8f6f4 (e4m3 x e4m3, fp32
// accumulate), four MMAs of K = 32 (+32 bytes = +2 in a descriptor's address field) from a fresh
// accumulator.  One block of instructions: the offsets are added inside, off the issuing lane's path.
MOE_DEVICE void mma_f8_block(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred f, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 f, %3, %3;\n\tsetp.eq.b32 t, %3, %3;\n\t"
      "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, t;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, t;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc)
      : "memory");
}

// The producer's copies, everything in shared memory by address (see bulk_load and tma_load_2d).
MOE_DEVICE void mbar_arrive_expect_tx_u32(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
MOE_DEVICE void bulk_load_u32(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}
MOE_DEVICE void tma_load_2d_u32(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}

// tcgen05.commit / mbarrier.test_wait on a barrier given by its shared-memory address.
MOE_DEVICE void mma_commit_u32(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
MOE_DEVICE bool mbar_test_u32(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Arrive on the mbarrier once this thread's cp.async copies so far have landed (counts as one of the
// barrier's expected arrivals).
MOE_DEVICE void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Lane 0 of a converged warp arrives, predicated inside the block: a branch around the arrival costs
// the epilogue's K loop about a tenth of its time.
MOE_DEVICE void mbar_arrive_lane0_u32(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(threadIdx.x & 31)
      : "memory");
}
MOE_DEVICE void mbar_arrive_lane0(uint64_t* bar) { mbar_arrive_lane0_u32(smem_u32(bar)); }
MOE_DEVICE bool mbar_try_wait_u32(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Two fp16 values, `lo` in the low half, rounded to nearest even; magnitudes beyond fp16 become its
// largest, NaN stays NaN.
MOE_DEVICE uint32_t f32x2_to_f16x2_sat(float lo, float hi) {
  uint32_t v;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
  return v;
}

// Instruction descriptor, kind::f8f6f4: D fp32 (bits 4-5 = 1), A and B e4m3 (bits 7-9 and 10-12 =
// 0), both K-major, N >> 3 in bits [17,23), M >> 4 in bits [24,29).
MOE_DEVICE uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) { return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24); }

// Wait for this thread's TMEM loads.  The scales pass through, so that no multiplication of a loaded
// value with them moves above it.
MOE_DEVICE void tmem_wait_ld(uint64_t& s0, uint64_t& s1) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+l"(s0), "+l"(s1) : : "memory");
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
