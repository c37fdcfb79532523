// tok[t] = sum_j w[t][j] * rows[inv[t][j]] (+ shared[t]) (rows.cuh).  Bound by memory: each row in
// expert order is read once, a token row written once (with dots: one more read).  The sum is taken
// in fp32 in slot order, the shared term last, and rounded once.
#include "rows.cuh"

namespace moe {

template <bool kVec>
MOE_DEVICE void add_shared(const RowsArgs& a, int64_t t, int col, int lane, float (&acc)[8]) {
  float f[8];
  if (a.shared_type == MOE_BF16) {
    Span<Bf16, kVec> s;
    s.load(static_cast<const Bf16*>(a.shared) + t * a.ld_shared, col, lane, a.d);
    s.to_f32(f);
  } else if (a.shared_type == MOE_FP16) {
    Span<Fp16, kVec> s;
    s.load(static_cast<const Fp16*>(a.shared) + t * a.ld_shared, col, lane, a.d);
    s.to_f32(f);
  } else {
    Span<Fp32, kVec> s;
    s.load(static_cast<const Fp32*>(a.shared) + t * a.ld_shared, col, lane, a.d);
    s.to_f32(f);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[q] += f[q];
}

// One slot group: the rows' loads first, then the sums (and the dots with xf).
template <typename ER, bool kVec, bool kDots>
MOE_DEVICE void add_slots(const RowsArgs& a, int col, int lane, const int (&r)[kSlots], const float (&w)[kSlots],
                          const float (&xf)[8], float (&sum)[8], float (&acc)[kSlots]) {
  Span<ER, kVec> z[kSlots];
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    if (r[u] >= 0)
      z[u].load(static_cast<const ER*>(a.rows) + r[u] * a.ld_rows, col, lane, a.d);
    else
      z[u].zero();
  }
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    if (r[u] < 0) continue;
    float zf[8];
    z[u].to_f32(zf);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      sum[q] = fmaf(w[u], zf[q], sum[q]);
      if (kDots) acc[u] = fmaf(xf[q], zf[q], acc[u]);
    }
  }
}

// Three blocks of 16-bit rows an SM, two of 32-bit ones (rows_spread.cu).  Gathering 8 rows a token with
// dots, 8195 tokens of 2048: 85 us with no bound, 67 with three; rows of 2047, not aligned: 592 and 152.
template <typename ET, typename ER, bool kVec, bool kDots>
__global__ void __launch_bounds__(kRowWarps * 32, sizeof(ER) == 2 ? 3 : 2) gather_kernel(const RowsArgs a) {
  __shared__ float part[kDots ? kRowWarps : 1][kSlots];
  pdl_trigger();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  ET* out = static_cast<ET*>(a.out) + t * a.ld_out;
  const ET* tok = static_cast<const ET*>(a.tok) + t * a.ld_tok;
  const int first = (blockIdx.y * warps + (threadIdx.x >> 5)) * kSpan, step = warps * gridDim.y * kSpan;
  int r[kSlots];
  float w[kSlots], acc[kSlots] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  load_slots(a, t, 0, r, w);
  for (int col = first; col < a.d; col += step) {
    float xf[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (kDots) {
      Span<ET, kVec> x;
      x.load(tok, col, lane, a.d);
      x.to_f32(xf);
    }
    add_slots<ER, kVec, kDots>(a, col, lane, r, w, xf, sum, acc);
    for (int j0 = kSlots; j0 < a.k; j0 += kSlots) {  // more than eight experts a token
      int r2[kSlots];
      float w2[kSlots], unused[kSlots];
      load_slots(a, t, j0, r2, w2);
      add_slots<ER, kVec, false>(a, col, lane, r2, w2, xf, sum, unused);
    }
    if (a.shared) add_shared<kVec>(a, t, col, lane, sum);
    Span<ET, kVec>::store(out, col, lane, a.d, sum);
  }
  if (kDots) {
    sum_dots(a, t, 0, r, acc, part);
    for (int j0 = kSlots; j0 < a.k; j0 += kSlots) {  // (the rows' second read comes from the caches)
      load_slots(a, t, j0, r, w);
#pragma unroll
      for (int u = 0; u < kSlots; ++u) acc[u] = 0.0f;
      for (int col = first; col < a.d; col += step) {
        float xf[8], unused[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        Span<ET, kVec> x;
        x.load(tok, col, lane, a.d);
        x.to_f32(xf);
        add_slots<ER, kVec, true>(a, col, lane, r, w, xf, unused, acc);
      }
      sum_dots(a, t, j0, r, acc, part);
    }
  }
}

template <typename ET, typename ER, bool kVec, bool kDots>
struct Gather {
  static void (*fn())(RowsArgs) { return gather_kernel<ET, ER, kVec, kDots>; }
};

cudaError_t launch_gather(const RowsArgs& a, moe_dtype tok, moe_dtype rows, bool vec, cudaStream_t st) {
  return launch_rows<Gather>(a, tok, rows, vec, st);
}

}  // namespace moe
