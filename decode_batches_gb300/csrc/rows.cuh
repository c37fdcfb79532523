// Rows in token order and rows in expert order.  inv[t][j] is the row, in expert order, of token
// t's assignment j (moe_permute's inv_perm; < 0: dropped).  Two kernels do all four directions:
//   spread   rows[inv[t][j]] = w[t][j] * tok[t]          (sort; the combine's gradient)
//   gather   tok[t] = sum_j w[t][j] * rows[inv[t][j]]    (combine; the sort's gradient)
// and, on request, dots[t][j] = <tok'[t], rows'[inv[t][j]]>, the weights' gradient, from the same
// pass.  Both go by tokens: a token's row is read (or written) once and its assignments' rows once
// each, so neither needs the forward permutation and nothing is read twice.
#pragma once

#include "abi_checks.h"
#include "elems.cuh"

namespace moe {

struct RowsArgs {
  const void* tok = nullptr;      // spread: the token rows; gather: the dots' token rows
  int64_t ld_tok = 0;
  const void* rows = nullptr;     // gather: the rows in expert order; spread: the dots' rows
  int64_t ld_rows = 0;
  const void* shared = nullptr;   // gather: a token row added last, or NULL
  int shared_type = MOE_FP32;
  int64_t ld_shared = 0;
  void* out = nullptr;            // spread: rows in expert order; gather: token rows
  int64_t ld_out = 0;
  const int32_t* inv = nullptr;   // [T][k]
  const float* w = nullptr;       // [T][k] or NULL (1)
  float* dots = nullptr;          // [T][k] or NULL
  int64_t n_rows = 0;             // entries of inv at or above it are treated like dropped ones
  int T = 0, k = 0, d = 0;
};

cudaError_t launch_spread(const RowsArgs& a, moe_dtype tok, moe_dtype rows, bool vec, cudaStream_t st);
cudaError_t launch_gather(const RowsArgs& a, moe_dtype tok, moe_dtype rows, bool vec, cudaStream_t st);

constexpr int kSlots = 8;          // assignments whose rows are in flight together
constexpr int kSpan = 256;         // columns a warp handles at a time: 8 a lane
constexpr int kRowWarps = 8;       // warps of a block, at most

// A lane's eight elements of a span: neighbours (16-byte accesses, rows and width aligned), or, where
// a row may start anywhere, every 32nd element, so that a warp's accesses stay contiguous.
template <typename E, bool kVec>
struct Span;

template <typename E>
struct Span<E, true> {
  Raw8<E> r;
  MOE_DEVICE void zero() { r.zero(); }
  MOE_DEVICE void load(const E* row, int col, int lane, int d) {
    if (col + lane * 8 < d)
      r.load(row + col + lane * 8);
    else
      r.zero();
  }
  MOE_DEVICE void to_f32(float (&o)[8]) const { r.to_f32(o); }
  static MOE_DEVICE void store(E* row, int col, int lane, int d, const float (&v)[8]) {
    if (col + lane * 8 < d) store8(row + col + lane * 8, v);
  }
  MOE_DEVICE void store_raw(E* row, int col, int lane, int d) const {
    if (col + lane * 8 < d) r.store(row + col + lane * 8);
  }
};

template <typename E>
struct Span<E, false> {
  E r[8];
  MOE_DEVICE void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = E{};
  }
  MOE_DEVICE void load(const E* row, int col, int lane, int d) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = col + 32 * i + lane < d ? row[col + 32 * i + lane] : E{};
  }
  MOE_DEVICE void to_f32(float (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = r[i].f32();
  }
  static MOE_DEVICE void store(E* row, int col, int lane, int d, const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + 32 * i + lane < d) row[col + 32 * i + lane] = E::of(v[i]);
  }
  MOE_DEVICE void store_raw(E* row, int col, int lane, int d) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + 32 * i + lane < d) row[col + 32 * i + lane] = r[i];
  }
};

// The rows and weights of slots j0 .. j0 + 7 of token t (-1 past the last, or dropped).
MOE_DEVICE void load_slots(const RowsArgs& a, int64_t t, int j0, int (&r)[kSlots], float (&w)[kSlots]) {
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    const bool in = j0 + u < a.k;
    const int v = in ? a.inv[t * a.k + j0 + u] : -1;
    r[u] = v < a.n_rows ? v : -1;
    w[u] = in && a.w ? a.w[t * a.k + j0 + u] : 1.0f;
  }
}

// acc[u] of all lanes and warps -> dots[t][j0 + u].  The order of the sums is fixed: pairs of lanes
// 16, 8, 4, 2, 1 apart, then the warps in order.  Every thread of the block calls it.
MOE_DEVICE void sum_dots(const RowsArgs& a, int64_t t, int j0, const int (&r)[kSlots], float (&acc)[kSlots],
                         float (*part)[kSlots]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int h = 4; h >= 1; h >>= 1) {  // halve the slots a lane holds: 8 -> 4 -> 2 -> 1
    const bool up = lane & (h * 4);
#pragma unroll
    for (int u = 0; u < h; ++u) {
      const float send = up ? acc[u] : acc[u + h], keep = up ? acc[u + h] : acc[u];
      acc[u] = keep + __shfl_xor_sync(0xffffffffu, send, h * 4);
    }
  }
  float s = acc[0];  // slot: bits 4, 3, 2 of the lane
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  if ((lane & 3) == 0) part[warp][lane >> 2] = s;
  __syncthreads();
  if (threadIdx.x < kSlots && j0 + threadIdx.x < a.k) {
    float v = 0.0f;
    for (int i = 0; i < warps; ++i) v += part[i][threadIdx.x];
    bool used = false;
#pragma unroll
    for (int u = 0; u < kSlots; ++u) used |= u == threadIdx.x && r[u] >= 0;
    a.dots[t * a.k + j0 + threadIdx.x] = used ? v : 0.0f;
  }
  if (j0 + kSlots < a.k) __syncthreads();
}

// Grid and block: with dots, a block holds a token's whole row (its sums meet in shared memory);
// without, a token's spans are spread over blocks of four warps, so that few tokens still fill SMs.
// A kernel whose blocks go on to further tokens (kBlocks of kRowWarps warps an SM, else 0) gets as many
// as fit at once, above four times as many tokens; below, the last tokens would wait for whole turns
// (517 tokens of 8 rows with dots: 4.6 us with a block a token, 5.0 in turns).
inline void rows_grid(const RowsArgs& a, int blocks, dim3* grid, dim3* block) {
  const int spans = (a.d + kSpan - 1) / kSpan;
  const int per = a.dots ? kRowWarps : 4, warps = spans < per ? spans : per;
  *block = dim3(32 * warps);
  *grid = dim3(a.T, a.dots ? 1 : (spans + warps - 1) / warps);
  if (blocks == 0) return;
  const int64_t need = static_cast<int64_t>(warps) * grid->y, fit = static_cast<int64_t>(current_sms()) * blocks * kRowWarps;
  const int64_t at_once = fit > need ? fit / need : 1;
  if (a.T > 4 * at_once) grid->x = static_cast<unsigned>(at_once);
}

template <template <typename, typename, bool, bool> class K, typename ET, typename ER, bool kVec, bool kDots>
cudaError_t launch_rows_as(const RowsArgs& a, cudaStream_t st) {
  dim3 grid, block;
  rows_grid(a, K<ET, ER, kVec, kDots>::kBlocks, &grid, &block);
  return launch_pdl(K<ET, ER, kVec, kDots>::fn(), grid, block, 0, st, a);
}

template <template <typename, typename, bool, bool> class K, bool kVec, bool kDots>
cudaError_t launch_rows_typed(const RowsArgs& a, moe_dtype tok, moe_dtype rows, cudaStream_t st) {
  switch (tok * 3 + rows) {
    case 0: return launch_rows_as<K, Bf16, Bf16, kVec, kDots>(a, st);
    case 1: return launch_rows_as<K, Bf16, Fp16, kVec, kDots>(a, st);
    case 2: return launch_rows_as<K, Bf16, Fp32, kVec, kDots>(a, st);
    case 3: return launch_rows_as<K, Fp16, Bf16, kVec, kDots>(a, st);
    case 4: return launch_rows_as<K, Fp16, Fp16, kVec, kDots>(a, st);
    case 5: return launch_rows_as<K, Fp16, Fp32, kVec, kDots>(a, st);
    case 6: return launch_rows_as<K, Fp32, Bf16, kVec, kDots>(a, st);
    case 7: return launch_rows_as<K, Fp32, Fp16, kVec, kDots>(a, st);
    default: return launch_rows_as<K, Fp32, Fp32, kVec, kDots>(a, st);
  }
}

template <template <typename, typename, bool, bool> class K>
cudaError_t launch_rows(const RowsArgs& a, moe_dtype tok, moe_dtype rows, bool vec, cudaStream_t st) {
  if (vec) return a.dots ? launch_rows_typed<K, true, true>(a, tok, rows, st) : launch_rows_typed<K, true, false>(a, tok, rows, st);
  return a.dots ? launch_rows_typed<K, false, true>(a, tok, rows, st) : launch_rows_typed<K, false, false>(a, tok, rows, st);
}

}  // namespace moe
