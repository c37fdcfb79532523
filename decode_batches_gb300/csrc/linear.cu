// C ABI of the 8-bit projection and of the quantisation calls (include/moe.h): handle, checks,
// weight set-up and the two launches of a call (quantise the rows, multiply).
#include <cudaTypedefs.h>

#include <cstdio>
#include <new>

#include "fp8.cuh"
#include "kernels.h"

using namespace moe;

struct moe_linear {
  int N = 0, K = 0, nk = 0, halves = 0;
  int num_sms = 1;
  uint8_t* w = nullptr;  // f8 tiles and their scales
  float* ws = nullptr;
  uint32_t* err = nullptr;
  bool weights_set = false;
  uint8_t* ws_ptr = nullptr;  // caller-owned workspace: codes [T][nk * 128], scales [T][f8_scale_ld(nk)]
  int T_max = 0;
};

static moe_status bad(moe_status s, const char* msg) { return fail_message(s, msg); }

static moe_status cuda_fail(const char* what, cudaError_t e) {
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", what, cudaGetErrorString(e));
  return fail_message(MOE_ERR_CUDA, buf);
}
#define LIN_TRY(expr)                                      \
  do {                                                     \
    const cudaError_t _e = (expr);                         \
    if (_e != cudaSuccess) return cuda_fail(#expr, _e);    \
  } while (0)

static bool known(moe_dtype t) { return t == MOE_BF16 || t == MOE_FP16 || t == MOE_FP32; }
static size_t elem_bytes(moe_dtype t) { return t == MOE_FP32 ? 4 : 2; }
static bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Rows and columns a call takes: an index past the end of a partial block or tile stays below 2^31.
constexpr int kMaxLen = 0x7fffffff - 2047;

static int current_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

extern "C" moe_status moe_quantize_rows(const void* x, moe_dtype x_dtype, int64_t ldx, int T, int K, uint8_t* q,
                                        int64_t ldq, float* s, int64_t lds, moe_stream_t stream) {
  if (T < 0 || K < 1) return bad(MOE_ERR_INVALID_ARG, "T must be >= 0 and K >= 1");
  if (!known(x_dtype)) return bad(MOE_ERR_INVALID_ARG, "unknown element type");
  if (K > kMaxLen) return bad(MOE_ERR_UNSUPPORTED, "at most 2^31 - 2048 columns");
  if (T == 0) return MOE_OK;
  if (!x || !q || !s) return bad(MOE_ERR_INVALID_ARG, "x, q and s are required");
  const int64_t nb = (K + kF8Block - 1) / kF8Block;
  if (ldx < K || ldq < nb * kF8Block || ldq % 16 || lds < nb)
    return bad(MOE_ERR_INVALID_ARG, "row pitches: ldx >= K, ldq >= K rounded up to 128 and a multiple of 16, lds >= ceil(K / 128)");
  if (!aligned(q, 16) || !aligned(x, elem_bytes(x_dtype)) || !aligned(s, 4))
    return bad(MOE_ERR_INVALID_ARG, "q must be 16-byte aligned, x and s aligned to their elements");
  LIN_TRY(launch_quant_rows(x, x_dtype, ldx, T, K, q, ldq, s, lds, current_sms(), reinterpret_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

extern "C" moe_status moe_quantize_blocks(const void* w, moe_dtype w_dtype, int rows, int K, uint8_t* q, float* s,
                                          moe_stream_t stream) {
  if (rows < 0 || K < 1) return bad(MOE_ERR_INVALID_ARG, "rows must be >= 0 and K >= 1");
  if (!known(w_dtype)) return bad(MOE_ERR_INVALID_ARG, "unknown element type");
  if (K > kMaxLen) return bad(MOE_ERR_UNSUPPORTED, "at most 2^31 - 2048 columns");
  if (rows == 0) return MOE_OK;
  if (!w || !q || !s) return bad(MOE_ERR_INVALID_ARG, "w, q and s are required");
  if (rows > 65535 * kF8Block) return bad(MOE_ERR_UNSUPPORTED, "at most 8388480 rows a call");
  LIN_TRY(launch_quant_blocks(w, w_dtype, K, rows, K, q, K, s, (K + kF8Block - 1) / kF8Block,
                              reinterpret_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

extern "C" moe_linear* moe_linear_create(int N, int K) {
  if (N < 1 || K < 1 || N > (1 << 20) || K > (1 << 20)) {
    bad(MOE_ERR_INVALID_ARG, "need 1 <= N, K <= 2^20");
    return nullptr;
  }
  moe_linear* l = new (std::nothrow) moe_linear();
  if (!l) {
    bad(MOE_ERR_CUDA, "out of host memory");
    return nullptr;
  }
  l->N = N;
  l->K = K;
  l->nk = (K + kF8Block - 1) / kF8Block;
  l->halves = f8_halves(N, false);
  l->num_sms = current_sms();
  fail_message(MOE_OK, "");
  return l;
}

extern "C" void moe_linear_destroy(moe_linear* l) {
  if (!l) return;
  if (l->w || l->err) cudaDeviceSynchronize();  // no queued work still reads the handle's memory
  cudaFree(l->w);
  cudaFree(l->ws);
  cudaFree(l->err);
  delete l;
}

extern "C" moe_status moe_linear_set_weights(moe_linear* l, const uint8_t* q, const float* s) {
  if (!l) return bad(MOE_ERR_INVALID_ARG, "the handle is NULL");
  if (!q || !s) return bad(MOE_ERR_INVALID_ARG, "q and s are required");
  LIN_TRY(cudaDeviceSynchronize());
  l->weights_set = false;
  if (!l->err) {
    LIN_TRY(cudaMalloc(&l->err, sizeof(uint32_t)));
    LIN_TRY(cudaMemset(l->err, 0, sizeof(uint32_t)));
  }
  const size_t tiles = (l->halves + 1) / 2;
  if (!l->w) LIN_TRY(cudaMalloc(&l->w, static_cast<size_t>(l->halves) * l->nk * kF8TileBytes));
  if (!l->ws) LIN_TRY(cudaMalloc(&l->ws, tiles * f8_scale_ld(l->nk) * 2 * sizeof(float)));
  LIN_TRY(launch_tile_fp8(q, s, nullptr, nullptr, l->w, l->ws, 1, l->N, l->K, 0));
  LIN_TRY(cudaDeviceSynchronize());
  l->weights_set = true;
  return MOE_OK;
}

static size_t codes_bytes(const moe_linear* l, int T) {
  return (static_cast<size_t>(T) * l->nk * kF8Block + 255) & ~size_t(255);
}

extern "C" size_t moe_linear_workspace_bytes(const moe_linear* l, int T_max) {
  if (!l || T_max < 0) return 0;
  const int T = T_max > 0 ? T_max : 1;
  return codes_bytes(l, T) + static_cast<size_t>(T) * f8_scale_ld(l->nk) * sizeof(float);
}

extern "C" moe_status moe_linear_set_workspace(moe_linear* l, void* dev_ptr, size_t bytes, int T_max) {
  if (!l) return bad(MOE_ERR_INVALID_ARG, "the handle is NULL");
  if (!dev_ptr || T_max < 1) return bad(MOE_ERR_INVALID_ARG, "workspace pointer and T_max >= 1 required");
  if (T_max > kMaxLen) return bad(MOE_ERR_UNSUPPORTED, "at most 2^31 - 2048 rows");
  if (!aligned(dev_ptr, 256)) return bad(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (bytes < moe_linear_workspace_bytes(l, T_max)) return bad(MOE_ERR_WORKSPACE, "workspace too small for T_max");
  l->ws_ptr = static_cast<uint8_t*>(dev_ptr);
  l->T_max = T_max;
  return MOE_OK;
}

static moe_status check_out(const moe_linear* l, int T, const void* out, moe_dtype out_dtype, int64_t ldo) {
  if (!l) return bad(MOE_ERR_INVALID_ARG, "the handle is NULL");
  if (T < 0) return bad(MOE_ERR_INVALID_ARG, "T must be >= 0");
  if (T > kMaxLen) return bad(MOE_ERR_UNSUPPORTED, "at most 2^31 - 2048 rows");
  if (!l->weights_set) return bad(MOE_ERR_NOT_READY, "weights not set");
  if (out_dtype != MOE_BF16 && out_dtype != MOE_FP32) return bad(MOE_ERR_INVALID_ARG, "out must be bf16 or fp32");
  if (T == 0) return MOE_OK;
  if (!out || ldo < l->N) return bad(MOE_ERR_INVALID_ARG, "out is required, with ldo >= N");
  if (!aligned(out, elem_bytes(out_dtype))) return bad(MOE_ERR_INVALID_ARG, "out must be aligned to its elements");
  return MOE_OK;
}

static moe_status product(moe_linear* l, const uint8_t* q, int64_t ldq, const float* s, int64_t lds, int T, void* out,
                          moe_dtype out_dtype, int64_t ldo, cudaStream_t st) {
  CUtensorMap m;
  F8Args a;
  // the rows are split into near-equal parts of at most 128: one box holds a part
  const int parts = (T + 127) / 128, most = (T + parts - 1) / parts;
  a.box_rows = (most + 31) / 32 * 32;
  moe_status r = make_map_f8(&m, q, l->K, T, ldq, a.box_rows);
  if (r != MOE_OK) return r;
  a.w = l->w;
  a.ws = l->ws;
  a.as = s;
  a.lds = lds;
  a.out = out;
  a.ldo = ldo;
  a.out_type = out_dtype;
  a.out_vec = aligned(out, 16) && (ldo * elem_bytes(out_dtype)) % 16 == 0 && (l->N * elem_bytes(out_dtype)) % 16 == 0;
  a.N = l->N;
  a.halves = l->halves;
  a.nk = l->nk;
  a.T = T;
  a.k = 1;
  a.err = l->err;
  CUtensorMap o{};  // (fewer than 32 rows never leave as a box)
  if (out_dtype == MOE_BF16 && a.out_vec && T >= 32 && (r = make_map_bf16_out(&o, out, l->N, T, ldo)) != MOE_OK) return r;
  LIN_TRY(launch_f8_linear(&m, &o, a, l->num_sms, st));
  return MOE_OK;
}

extern "C" moe_status moe_linear_forward(moe_linear* l, const void* x, moe_dtype x_dtype, int64_t ldx, int T, void* out,
                                         moe_dtype out_dtype, int64_t ldo, moe_stream_t stream) {
  moe_status r = check_out(l, T, out, out_dtype, ldo);
  if (r != MOE_OK) return r;
  if (!known(x_dtype)) return bad(MOE_ERR_INVALID_ARG, "unknown element type");
  if (T == 0) return MOE_OK;
  if (!l->ws_ptr) return bad(MOE_ERR_NOT_READY, "workspace not set");
  if (T > l->T_max) return bad(MOE_ERR_WORKSPACE, "T exceeds the workspace's T_max");
  if (!x || ldx < l->K) return bad(MOE_ERR_INVALID_ARG, "x is required, with ldx >= K");
  if (!aligned(x, elem_bytes(x_dtype))) return bad(MOE_ERR_INVALID_ARG, "x must be aligned to its elements");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* q = l->ws_ptr;
  float* s = reinterpret_cast<float*>(l->ws_ptr + codes_bytes(l, l->T_max));
  const int64_t ldq = static_cast<int64_t>(l->nk) * kF8Block, lds = f8_scale_ld(l->nk);
  LIN_TRY(launch_quant_rows(x, x_dtype, ldx, T, l->K, q, ldq, s, lds, l->num_sms, st));
  return product(l, q, ldq, s, lds, T, out, out_dtype, ldo, st);
}

extern "C" moe_status moe_linear_forward_quantized(moe_linear* l, const uint8_t* q, int64_t ldq, const float* s,
                                                   int64_t lds, int T, void* out, moe_dtype out_dtype, int64_t ldo,
                                                   moe_stream_t stream) {
  moe_status r = check_out(l, T, out, out_dtype, ldo);
  if (r != MOE_OK) return r;
  if (T == 0) return MOE_OK;
  if (!q || !s || ldq < l->K || ldq % 16 || lds < l->nk || lds % 4)
    return bad(MOE_ERR_INVALID_ARG, "q and s are required: ldq >= K and a multiple of 16, lds >= ceil(K / 128) and a multiple of 4");
  if (!aligned(q, 16) || !aligned(s, 16)) return bad(MOE_ERR_INVALID_ARG, "q and s must be 16-byte aligned");
  return product(l, q, ldq, s, lds, T, out, out_dtype, ldo, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_linear_get_device_error(moe_linear* l, uint32_t* code) {
  if (!l || !code) return bad(MOE_ERR_INVALID_ARG, "the handle and code are required");
  *code = 0;
  LIN_TRY(cudaDeviceSynchronize());
  if (!l->err) return MOE_OK;
  LIN_TRY(cudaMemcpy(code, l->err, sizeof(uint32_t), cudaMemcpyDeviceToHost));
  LIN_TRY(cudaMemset(l->err, 0, sizeof(uint32_t)));
  LIN_TRY(cudaDeviceSynchronize());  // cleared before a later call, on any stream, sets a bit
  return *code ? bad(MOE_ERR_DEVICE, "device error bits are set") : MOE_OK;
}
