// tok[t] = sum_j w[t][j] * rows[inv[t][j]] (+ shared[t]) (rows.cuh).  Bound by memory: each row in
// expert order is read once, a token row written once (with dots: one more read).  The sum is taken
// in fp32 in slot order, the shared term last, and rounded once.
#include "rows.cuh"

namespace moe {

// The shared term's eight elements: requested with the rows, added behind them.
template <bool kVec>
struct SharedSpan {
  union {
    Span<Bf16, kVec> b;
    Span<Fp16, kVec> h;
    Span<Fp32, kVec> f;
  };
  MOE_DEVICE SharedSpan() {}
  MOE_DEVICE void load(const RowsArgs& a, int64_t t, int col, int lane) {
    if (a.shared_type == MOE_BF16)
      b.load(static_cast<const Bf16*>(a.shared) + t * a.ld_shared, col, lane, a.d);
    else if (a.shared_type == MOE_FP16)
      h.load(static_cast<const Fp16*>(a.shared) + t * a.ld_shared, col, lane, a.d);
    else
      f.load(static_cast<const Fp32*>(a.shared) + t * a.ld_shared, col, lane, a.d);
  }
  MOE_DEVICE void add(const RowsArgs& a, float (&acc)[8]) const {
    float v[8];
    if (a.shared_type == MOE_BF16)
      b.to_f32(v);
    else if (a.shared_type == MOE_FP16)
      h.to_f32(v);
    else
      f.to_f32(v);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += v[q];
  }
};

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

// A lane's slot of token t: one load for the warp, handed round with shuffles.
MOE_DEVICE void slot_of(const RowsArgs& a, int64_t t, int lane, int& r, float& w) {
  const bool in = lane < kSlots && lane < a.k;
  const int v = in ? a.inv[t * a.k + lane] : -1;
  r = v < a.n_rows ? v : -1;
  w = in && a.w ? a.w[t * a.k + lane] : 1.0f;
}

// Blocks an SM: four of aligned 16-bit rows without dots, three of other 16-bit rows, two of 32-bit ones,
// so that enough loads are under way (no bound, four: 8195 tokens of 8 rows of 2048, 49.7 and 46.5 us;
// with dots no bound, three: 85 and 67; rows of 2047, not aligned: 592 and 152).
template <typename ER, bool kVec, bool kDots>
constexpr int kGatherBlocks = sizeof(ER) == 2 ? (kVec && !kDots ? 4 : 3) : 2;

// A block takes tokens gridDim.x apart and asks for the next one's slots before it sums this one, so
// that a token does not wait for them first: combine of 8195 tokens, top 6, 4096 columns, 88 us with a
// block a token, 79.5 so; with dots 66 and 56.5.
template <typename ET, typename ER, bool kVec, bool kDots>
__global__ void __launch_bounds__(kRowWarps * 32, kGatherBlocks<ER, kVec, kDots>) gather_kernel(const RowsArgs a) {
  __shared__ float part[kDots ? 2 : 1][kDots ? kRowWarps : 1][kSlots];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int first = (blockIdx.y * warps + (threadIdx.x >> 5)) * kSpan, step = warps * gridDim.y * kSpan;
  int next_r, turn = 0;
  float next_w;
  slot_of(a, blockIdx.x, lane, next_r, next_w);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    ET* out = static_cast<ET*>(a.out) + t * a.ld_out;
    const ET* tok = static_cast<const ET*>(a.tok) + t * a.ld_tok;
    int r[kSlots];
    float w[kSlots], acc[kSlots] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      r[u] = __shfl_sync(0xffffffffu, next_r, u);
      w[u] = __shfl_sync(0xffffffffu, next_w, u);
    }
    if (t + gridDim.x < a.T) slot_of(a, t + gridDim.x, lane, next_r, next_w);
    for (int col = first; col < a.d; col += step) {
      float xf[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (kDots) {
        Span<ET, kVec> x;
        x.load(tok, col, lane, a.d);
        x.to_f32(xf);
      }
      SharedSpan<kVec> sh;
      if (!kDots && a.shared) sh.load(a, t, col, lane);
      add_slots<ER, kVec, kDots>(a, col, lane, r, w, xf, sum, acc);
      for (int j0 = kSlots; j0 < a.k; j0 += kSlots) {  // more than eight experts a token
        int r2[kSlots];
        float w2[kSlots], unused[kSlots];
        load_slots(a, t, j0, r2, w2);
        add_slots<ER, kVec, false>(a, col, lane, r2, w2, xf, sum, unused);
      }
      if (!kDots && a.shared) sh.add(a, sum);
      Span<ET, kVec>::store(out, col, lane, a.d, sum);
    }
    if (kDots) {  // (the sums of two turns are held apart: a warp may be one barrier ahead)
      sum_dots(a, t, 0, r, acc, part[turn & 1]);
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
        sum_dots(a, t, j0, r, acc, part[turn & 1]);
      }
      ++turn;
    }
  }
}

template <typename ET, typename ER, bool kVec, bool kDots>
struct Gather {
  static constexpr int kBlocks = kGatherBlocks<ER, kVec, kDots>;
  static void (*fn())(RowsArgs) { return gather_kernel<ET, ER, kVec, kDots>; }
};

cudaError_t launch_gather(const RowsArgs& a, moe_dtype tok, moe_dtype rows, bool vec, cudaStream_t st) {
  return launch_rows<Gather>(a, tok, rows, vec, st);
}

}  // namespace moe
