// Element types of a call's tensors: eight neighbouring elements as fp32 values and back, one
// rounding to nearest even (out-of-range fp16 values become infinities).
#pragma once

#include "common.cuh"

namespace moe {

struct Bf16 {
  uint16_t v;
  MOE_DEVICE float f32() const { return bf16_bits_to_f32(v); }
  static MOE_DEVICE Bf16 of(float f) { return Bf16{f32_to_bf16_bits_rn(f)}; }
};
struct Fp16 {
  uint16_t v;
  MOE_DEVICE float f32() const { return f16_bits_to_f32(v); }
  static MOE_DEVICE Fp16 of(float f) { return Fp16{f32_to_f16_bits_rn(f)}; }
};
struct Fp32 {
  float v;
  MOE_DEVICE float f32() const { return v; }
  static MOE_DEVICE Fp32 of(float f) { return Fp32{f}; }
};

MOE_DEVICE uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight elements as loaded: requested early, converted where they are used.
template <typename E>
struct Raw8 {
  uint4 a;
  MOE_DEVICE void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  MOE_DEVICE void load(const E* p) { a = *reinterpret_cast<const uint4*>(p); }
  MOE_DEVICE void store(E* p) const { *reinterpret_cast<uint4*>(p) = a; }
  MOE_DEVICE void to_f32(float (&o)[8]) const;
};
template <>
MOE_DEVICE void Raw8<Bf16>::to_f32(float (&o)[8]) const { bf16x8_to_f32(a, o); }
template <>
MOE_DEVICE void Raw8<Fp16>::to_f32(float (&o)[8]) const { f16x8_to_f32(a, o); }
template <>
struct Raw8<Fp32> {
  uint4 a, b;
  MOE_DEVICE void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  MOE_DEVICE void load(const Fp32* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  MOE_DEVICE void store(Fp32* p) const {
    reinterpret_cast<uint4*>(p)[0] = a;
    reinterpret_cast<uint4*>(p)[1] = b;
  }
  MOE_DEVICE void to_f32(float (&o)[8]) const {
    o[0] = __uint_as_float(a.x), o[1] = __uint_as_float(a.y), o[2] = __uint_as_float(a.z), o[3] = __uint_as_float(a.w);
    o[4] = __uint_as_float(b.x), o[5] = __uint_as_float(b.y), o[6] = __uint_as_float(b.z), o[7] = __uint_as_float(b.w);
  }
};

// (cvt.rn.bf16x2 takes the upper half first)
MOE_DEVICE uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
MOE_DEVICE void store8(Bf16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]),
                                            cvt_bf16x2(v[6], v[7]));
}
MOE_DEVICE void store8(Fp16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                                            pack_f16x2(v[6], v[7]));
}
MOE_DEVICE void store8(Fp32* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// v += f, in pairs (each sum rounded as by itself)
MOE_DEVICE void add8(float (&v)[8], const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(v[i]), "+f"(v[i + 1])
        : "f"(f[i]), "f"(f[i + 1]));
}

}  // namespace moe
