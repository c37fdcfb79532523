// rows[inv[t][j]] = w[t][j] * tok[t] (rows.cuh).  Bound by memory: a token row is read once, each of
// its k rows written once (with dots: read once too).  Without weights and with one element type the
// bits are copied as they are.
#include <type_traits>

#include "rows.cuh"

namespace moe {

// Three blocks of aligned 16-bit rows an SM, two of all others, so that enough loads are under way.
// Spreading with dots and weights, 8195 tokens of 4096, top 6: bf16 148 us with no bound, 133 with
// three; fp16 rows of fp32 tokens 236 and 140.  4095 columns, not aligned: 517 us with one block, 300
// with two, 396 with three.
template <typename ET, typename ER, bool kVec, bool kDots>
__global__ void __launch_bounds__(kRowWarps * 32, kVec && sizeof(ER) == 2 ? 3 : 2) spread_kernel(const RowsArgs a) {
  __shared__ float part[kDots ? kRowWarps : 1][kSlots];
  pdl_trigger();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const ET* tok = static_cast<const ET*>(a.tok) + t * a.ld_tok;
  const int first = (blockIdx.y * warps + (threadIdx.x >> 5)) * kSpan, step = warps * gridDim.y * kSpan;
  for (int j0 = 0; j0 < a.k; j0 += kSlots) {
    int r[kSlots];
    float w[kSlots];
    load_slots(a, t, j0, r, w);
    float acc[kSlots] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int col = first; col < a.d; col += step) {
      Span<ET, kVec> x;
      Span<ER, kVec> z[kDots ? kSlots : 1];
      x.load(tok, col, lane, a.d);
      if (kDots) {
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
          if (r[u] >= 0)
            z[u].load(static_cast<const ER*>(a.rows) + r[u] * a.ld_rows, col, lane, a.d);
          else
            z[u].zero();
        }
      }
      float xf[8];
      x.to_f32(xf);
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        if (r[u] < 0) continue;
        ER* out = static_cast<ER*>(a.out) + r[u] * a.ld_out;
        if (std::is_same<ET, ER>::value && !a.w) {
          reinterpret_cast<const Span<ER, kVec>&>(x).store_raw(out, col, lane, a.d);
        } else {
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = w[u] * xf[q];
          Span<ER, kVec>::store(out, col, lane, a.d, v);
        }
        if (kDots) {
          float zf[8];
          z[u].to_f32(zf);
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[u] = fmaf(xf[q], zf[q], acc[u]);
        }
      }
    }
    if (kDots) sum_dots(a, t, j0, r, acc, part);
  }
}

template <typename ET, typename ER, bool kVec, bool kDots>
struct Spread {
  static constexpr int kBlocks = 0;  // a block a token
  static void (*fn())(RowsArgs) { return spread_kernel<ET, ER, kVec, kDots>; }
};

cudaError_t launch_spread(const RowsArgs& a, moe_dtype tok, moe_dtype rows, bool vec, cudaStream_t st) {
  return launch_rows<Spread>(a, tok, rows, vec, st);
}

}  // namespace moe
