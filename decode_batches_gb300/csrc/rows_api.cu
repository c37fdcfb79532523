// C ABI of the row moves between token order and expert order (include/moe.h): checks and launches.
#include "abi_checks.h"
#include "rows.cuh"

using namespace moe;

namespace {

struct Tensor {
  const void* p;
  moe_dtype type;
  int64_t ld, rows;
};

moe_status check_sizes(int T, int k, int d, int64_t n_rows) {
  if (T < 0 || k < 1 || k > 32 || d < 1 || n_rows < 0)
    return bad(MOE_ERR_INVALID_ARG, "need T >= 0, 1 <= k <= 32, d >= 1, n_rows >= 0");
  if (static_cast<int64_t>(T) * k > 0x7fffffff || d > (1 << 24) || n_rows > 0x7fffffff)
    return bad(MOE_ERR_UNSUPPORTED, "at most 2^31 - 1 assignments and rows of 2^24 columns");
  return MOE_OK;
}

moe_status check_tensor(const Tensor& t, int d) {
  if (!known(t.type)) return bad(MOE_ERR_INVALID_ARG, "unknown element type");
  if (!t.p) return bad(MOE_ERR_INVALID_ARG, "a required tensor is NULL");
  if (t.ld < d) return bad(MOE_ERR_INVALID_ARG, "a row pitch is below d");
  if (!aligned(t.p, elem_bytes(t.type))) return bad(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  return MOE_OK;
}

moe_status check_assignments(const int32_t* inv, const float* w, const float* dw) {
  if (!inv) return bad(MOE_ERR_INVALID_ARG, "inv_perm is required");
  if (!aligned(inv, 4) || !aligned(w, 4) || !aligned(dw, 4))
    return bad(MOE_ERR_INVALID_ARG, "inv_perm, weights and dweights must be aligned to their elements");
  return MOE_OK;
}

bool vectors(const Tensor& t, int d) { return d % 8 == 0 && rows_aligned16(t.p, t.ld, t.type, t.rows); }

}  // namespace

#define ROWS_TRY(expr)                 \
  do {                                 \
    const moe_status _s = (expr);      \
    if (_s != MOE_OK) return _s;       \
  } while (0)

extern "C" moe_status moe_sort_rows(const void* x, moe_dtype x_dtype, int64_t ldx, int T, int k, int d,
                                    const int32_t* inv_perm, const float* weights, void* out, int64_t ldo,
                                    int64_t n_rows, moe_stream_t stream) {
  ROWS_TRY(check_sizes(T, k, d, n_rows));
  if (T == 0 || n_rows == 0) return MOE_OK;
  const Tensor tok{x, x_dtype, ldx, T}, rows{out, x_dtype, ldo, n_rows};
  ROWS_TRY(check_tensor(tok, d));
  ROWS_TRY(check_tensor(rows, d));
  ROWS_TRY(check_assignments(inv_perm, weights, nullptr));
  RowsArgs a;
  a.tok = x, a.ld_tok = ldx, a.out = out, a.ld_out = ldo;
  a.inv = inv_perm, a.w = weights, a.n_rows = n_rows, a.T = T, a.k = k, a.d = d;
  LIN_TRY(launch_spread(a, x_dtype, x_dtype, vectors(tok, d) && vectors(rows, d), reinterpret_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

extern "C" moe_status moe_sort_rows_backward(const void* grad, moe_dtype dtype, int64_t ldg, int64_t n_rows, int T, int k,
                                             int d, const int32_t* inv_perm, const float* weights, const void* x,
                                             int64_t ldx, void* dx, int64_t lddx, float* dweights, moe_stream_t stream) {
  ROWS_TRY(check_sizes(T, k, d, n_rows));
  if (T == 0) return MOE_OK;
  const Tensor rows{grad, dtype, ldg, n_rows}, tok{x, dtype, ldx, T}, out{dx, dtype, lddx, T};
  if (n_rows > 0) ROWS_TRY(check_tensor(rows, d));
  ROWS_TRY(check_tensor(out, d));
  if (dweights) ROWS_TRY(check_tensor(tok, d));
  ROWS_TRY(check_assignments(inv_perm, weights, dweights));
  RowsArgs a;
  a.tok = x, a.ld_tok = ldx, a.rows = grad, a.ld_rows = ldg, a.out = dx, a.ld_out = lddx;
  a.inv = inv_perm, a.w = weights, a.dots = dweights, a.n_rows = n_rows, a.T = T, a.k = k, a.d = d;
  const bool vec = vectors(rows, d) && vectors(out, d) && (!dweights || vectors(tok, d));
  LIN_TRY(launch_gather(a, dtype, dtype, vec, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

extern "C" moe_status moe_combine_rows(const void* y, moe_dtype y_dtype, int64_t ldy, int64_t n_rows, int T, int k, int d,
                                       const int32_t* inv_perm, const float* weights, const void* shared,
                                       moe_dtype shared_dtype, int64_t lds, void* out, moe_dtype out_dtype, int64_t ldo,
                                       moe_stream_t stream) {
  ROWS_TRY(check_sizes(T, k, d, n_rows));
  if (T == 0) return MOE_OK;
  const Tensor rows{y, y_dtype, ldy, n_rows}, add{shared, shared_dtype, lds, T}, res{out, out_dtype, ldo, T};
  if (!known(y_dtype)) return bad(MOE_ERR_INVALID_ARG, "unknown element type");
  if (n_rows > 0) ROWS_TRY(check_tensor(rows, d));
  ROWS_TRY(check_tensor(res, d));
  if (shared) ROWS_TRY(check_tensor(add, d));
  ROWS_TRY(check_assignments(inv_perm, weights, nullptr));
  RowsArgs a;
  a.rows = y, a.ld_rows = ldy, a.shared = shared, a.shared_type = shared_dtype, a.ld_shared = lds;
  a.out = out, a.ld_out = ldo, a.inv = inv_perm, a.w = weights, a.n_rows = n_rows, a.T = T, a.k = k, a.d = d;
  const bool vec = vectors(rows, d) && vectors(res, d) && (!shared || vectors(add, d));
  LIN_TRY(launch_gather(a, out_dtype, y_dtype, vec, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

extern "C" moe_status moe_combine_rows_backward(const void* grad, moe_dtype grad_dtype, int64_t ldg, int T, int k, int d,
                                                const int32_t* inv_perm, const float* weights, const void* y, int64_t ldy,
                                                void* dy, moe_dtype y_dtype, int64_t lddy, int64_t n_rows,
                                                float* dweights, moe_stream_t stream) {
  ROWS_TRY(check_sizes(T, k, d, n_rows));
  if (T == 0) return MOE_OK;
  const Tensor tok{grad, grad_dtype, ldg, T}, rows{y, y_dtype, ldy, n_rows}, out{dy, y_dtype, lddy, n_rows};
  ROWS_TRY(check_tensor(tok, d));
  if (!known(y_dtype)) return bad(MOE_ERR_INVALID_ARG, "unknown element type");
  if (n_rows > 0) ROWS_TRY(check_tensor(out, d));
  if (dweights && n_rows > 0) ROWS_TRY(check_tensor(rows, d));
  ROWS_TRY(check_assignments(inv_perm, weights, dweights));
  RowsArgs a;
  a.tok = grad, a.ld_tok = ldg, a.rows = y, a.ld_rows = ldy, a.out = dy, a.ld_out = lddy;
  a.inv = inv_perm, a.w = weights, a.dots = dweights, a.n_rows = n_rows, a.T = T, a.k = k, a.d = d;
  const bool vec = vectors(tok, d) && vectors(out, d) && (!dweights || vectors(rows, d));
  LIN_TRY(launch_spread(a, grad_dtype, y_dtype, vec, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_OK;
}
