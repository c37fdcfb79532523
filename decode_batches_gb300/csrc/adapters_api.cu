// C ABI of the low-rank adapters (include/moe.h): handle, slots, checks and the launches of a call.
#include <new>

#include "abi_checks.h"
#include "adapters.cuh"

using namespace moe;

struct moe_adapters {
  int n = 0, N = 0, K = 0, r = 0, rpad = 0;
  moe_dtype type = MOE_BF16;
  int num_sms = 1;           // of the handle's device (before there is one: of the current at create)
  int device = -1;           // of the handle's memory, once there is any
  uint16_t* w = nullptr;     // packed weights: A of all slots, B, and both again as the tensor cores' tiles
  int32_t* rank = nullptr;   // [n]
  float* scale = nullptr;    // [n]
  uint32_t* err = nullptr;
  uint8_t* ws = nullptr;     // caller-owned: tile count, tiles, order
  int T_max = 0;
  int64_t a_slot() const { return adapter_a_elems(K, rpad); }
  int64_t b_slot() const { return adapter_b_elems(N, rpad); }
  int64_t a_tc_slot() const { return adapter_tc_a_elems(K, rpad); }
  int64_t b_tc_slot() const { return adapter_tc_b_elems(N, rpad); }
  int64_t slot_elems() const { return a_slot() + b_slot() + a_tc_slot() + b_tc_slot(); }
  uint16_t* a() const { return w; }
  uint16_t* b() const { return a() + n * a_slot(); }
  uint16_t* a_tc() const { return b() + n * b_slot(); }
  uint16_t* b_tc() const { return a_tc() + n * a_tc_slot(); }
};

constexpr int kMaxRows = 1 << 26;

static size_t tile_bytes(const moe_adapters* h, int T) {
  // an entry for every cluster of a grid: whole waves beside T / 128 + n tiles, and those that copy
  return (static_cast<size_t>(T / kAdapterTileRows + h->n + 4 + 4 * h->num_sms) * sizeof(AdapterTile) + 255) & ~size_t(255);
}

extern "C" moe_adapters* moe_adapters_create(int n, int N, int K, int r_max, moe_dtype dtype) {
  if (n < 1 || n > kAdaptersMax || N < 1 || K < 1 || N > (1 << 20) || K > (1 << 20) || r_max < 1 ||
      r_max > kAdapterRankMax || (dtype != MOE_BF16 && dtype != MOE_FP16)) {
    bad(MOE_ERR_INVALID_ARG, "need 1 <= n <= 1024, 1 <= N, K <= 2^20, 1 <= r_max <= 128, bf16 or fp16");
    return nullptr;
  }
  moe_adapters* h = new (std::nothrow) moe_adapters();
  if (!h) {
    bad(MOE_ERR_CUDA, "out of host memory");
    return nullptr;
  }
  h->n = n, h->N = N, h->K = K, h->r = r_max, h->rpad = adapter_rank_pad(r_max), h->type = dtype;
  h->num_sms = current_sms();
  fail_message(MOE_OK, "");
  return h;
}

extern "C" void moe_adapters_destroy(moe_adapters* h) {
  if (!h) return;
  if (h->w || h->rank || h->scale || h->err) cudaDeviceSynchronize();  // no queued work still reads the handle's memory
  cudaFree(h->w);
  cudaFree(h->rank);
  cudaFree(h->scale);
  cudaFree(h->err);
  delete h;
}

// The slots' memory, all empty, on the first slot that is set or the workspace, whichever comes first.
static moe_status allocate(moe_adapters* h) {
  const int dev = current_device();
  if (h->device >= 0 && h->device != dev)
    return bad(MOE_ERR_INVALID_ARG, "the handle's memory is on another device than the current one");
  if (h->device < 0) h->num_sms = current_sms();
  h->device = dev;
  if (!h->err) {
    LIN_TRY(cudaMalloc(&h->err, sizeof(uint32_t)));
    LIN_TRY(cudaMemset(h->err, 0, sizeof(uint32_t)));
  }
  if (!h->scale) LIN_TRY(cudaMalloc(&h->scale, h->n * sizeof(float)));
  if (!h->w) LIN_TRY(cudaMalloc(&h->w, static_cast<size_t>(h->n) * h->slot_elems() * sizeof(uint16_t)));
  if (!h->rank) {
    int32_t* p = nullptr;
    LIN_TRY(cudaMalloc(&p, h->n * sizeof(int32_t)));
    const cudaError_t e = cudaMemset(p, 0, h->n * sizeof(int32_t));
    if (e != cudaSuccess) {
      cudaFree(p);
      return cuda_fail("cudaMemset", e);
    }
    h->rank = p;
  }
  LIN_TRY(cudaDeviceSynchronize());
  return MOE_OK;
}

extern "C" moe_status moe_adapters_set(moe_adapters* h, int slot, const void* a, const void* b, int r, float scale) {
  if (!h) return bad(MOE_ERR_INVALID_ARG, "the handle is NULL");
  if (slot < 0 || slot >= h->n) return bad(MOE_ERR_INVALID_ARG, "slot outside [0, n)");
  if (r < 0 || r > h->r) return bad(MOE_ERR_INVALID_ARG, "need 0 <= r <= r_max");
  if (r > 0 && (!a || !b)) return bad(MOE_ERR_INVALID_ARG, "a and b are required");
  if (!aligned(a, 2) || !aligned(b, 2)) return bad(MOE_ERR_INVALID_ARG, "a and b must be aligned to their elements");
  if (!(scale - scale == 0.0f)) return bad(MOE_ERR_INVALID_ARG, "scale must be finite");
  const moe_status s = allocate(h);
  if (s != MOE_OK) return s;
  LIN_TRY(cudaDeviceSynchronize());  // queued calls still use the slot's old contents
  // (the slot is empty until all of it is written)
  LIN_TRY(cudaMemset(h->rank + slot, 0, sizeof(int32_t)));
  if (r > 0) {
    const uint16_t *pa = static_cast<const uint16_t*>(a), *pb = static_cast<const uint16_t*>(b);
    LIN_TRY(launch_adapter_pack(pa, pb, h->a() + slot * h->a_slot(), h->b() + slot * h->b_slot(), r, h->K, h->N, h->rpad, 0));
    LIN_TRY(launch_adapter_tc_pack(pa, pb, h->a_tc() + slot * h->a_tc_slot(), h->b_tc() + slot * h->b_tc_slot(), r, h->K,
                                   h->N, h->rpad, 0));
    LIN_TRY(cudaMemcpy(h->scale + slot, &scale, sizeof scale, cudaMemcpyHostToDevice));
    LIN_TRY(cudaDeviceSynchronize());
    LIN_TRY(cudaMemcpy(h->rank + slot, &r, sizeof(int32_t), cudaMemcpyHostToDevice));
  }
  LIN_TRY(cudaDeviceSynchronize());
  return MOE_OK;
}

extern "C" size_t moe_adapters_workspace_bytes(const moe_adapters* h, int T_max) {
  if (!h || T_max < 0) return 0;
  const int T = T_max > 0 ? T_max : 1;
  return 256 + tile_bytes(h, T) + static_cast<size_t>(T) * sizeof(int32_t);
}

extern "C" moe_status moe_adapters_set_workspace(moe_adapters* h, void* dev_ptr, size_t bytes, int T_max) {
  if (!h) return bad(MOE_ERR_INVALID_ARG, "the handle is NULL");
  if (!dev_ptr || T_max < 1) return bad(MOE_ERR_INVALID_ARG, "workspace pointer and T_max >= 1 required");
  if (T_max > kMaxRows) return bad(MOE_ERR_UNSUPPORTED, "at most 2^26 rows");
  if (!aligned(dev_ptr, 256)) return bad(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (bytes < moe_adapters_workspace_bytes(h, T_max)) return bad(MOE_ERR_WORKSPACE, "workspace too small for T_max");
  const moe_status s = allocate(h);
  if (s != MOE_OK) return s;
  // (again: the handle's device, known now, may have more SMs than that of create)
  if (bytes < moe_adapters_workspace_bytes(h, T_max)) return bad(MOE_ERR_WORKSPACE, "workspace too small for T_max");
  h->ws = static_cast<uint8_t*>(dev_ptr);
  h->T_max = T_max;
  return MOE_OK;
}

extern "C" moe_status moe_adapters_forward(moe_adapters* h, const void* x, int64_t ldx, int T, const int32_t* ids,
                                           const void* base, int64_t ldb, void* out, moe_dtype out_dtype, int64_t ldo,
                                           moe_stream_t stream) {
  if (!h) return bad(MOE_ERR_INVALID_ARG, "the handle is NULL");
  if (T < 0) return bad(MOE_ERR_INVALID_ARG, "T must be >= 0");
  if (!known(out_dtype)) return bad(MOE_ERR_INVALID_ARG, "unknown element type");
  if (!h->ws) return bad(MOE_ERR_NOT_READY, "workspace not set");
  if (T > h->T_max) return bad(MOE_ERR_WORKSPACE, "T exceeds the workspace's T_max");
  if (T == 0) return MOE_OK;
  if (h->device != current_device())
    return bad(MOE_ERR_INVALID_ARG, "the handle's memory is on another device than the current one");
  if (!x || !ids || !out) return bad(MOE_ERR_INVALID_ARG, "x, ids and out are required");
  if (ldx < h->K || ldo < h->N || (base && ldb < h->N)) return bad(MOE_ERR_INVALID_ARG, "a row pitch is below the width");
  const size_t e = elem_bytes(out_dtype);
  if (!aligned(x, 2) || !aligned(ids, 4) || !aligned(out, e) || !aligned(base, e))
    return bad(MOE_ERR_INVALID_ARG, "x, ids, base and out must be aligned to their elements");
  if (base == out && ldb != ldo) return bad(MOE_ERR_INVALID_ARG, "base and out are the same rows: their pitches must be equal");
  AdapterArgs a;
  a.x = static_cast<const uint16_t*>(x), a.ldx = ldx, a.ids = ids;
  a.a = h->a(), a.b = h->b(), a.a_slot = h->a_slot(), a.b_slot = h->b_slot();
  a.a_tc = h->a_tc(), a.b_tc = h->b_tc(), a.a_tc_slot = h->a_tc_slot(), a.b_tc_slot = h->b_tc_slot();
  a.slots = AdapterSlots{h->rank, h->scale};
  a.base = base, a.ld_base = ldb, a.out = out, a.ld_out = ldo, a.out_type = out_dtype;
  a.x_vec = h->K % 8 == 0 && rows_aligned16(x, ldx, h->type, T);
  a.out_vec = h->N % 8 == 0 && rows_aligned16(out, ldo, out_dtype, T) && (!base || rows_aligned16(base, ldb, out_dtype, T));
  a.T = T, a.n = h->n, a.K = h->K, a.N = h->N, a.err = h->err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T <= kAdapterScan) {
    LIN_TRY(launch_adapters(a, h->rpad, h->type == MOE_FP16, h->num_sms, st));
    return MOE_OK;
  }
  a.cut = adapter_cut(T, h->n, h->rpad, h->num_sms);
  if (T > kAdapterCount) {
    a.cut.rows = kAdapterTileRows;  // (the grouping lowers it)
    int32_t* n_tiles = reinterpret_cast<int32_t*>(h->ws);
    AdapterTile* tiles = reinterpret_cast<AdapterTile*>(h->ws + 256);
    int32_t* order = reinterpret_cast<int32_t*>(h->ws + 256 + tile_bytes(h, h->T_max));
    LIN_TRY(launch_adapter_group(ids, T, h->n, a.cut, a.slots, order, tiles, n_tiles, h->err, st));
    a.order = order, a.tiles = tiles, a.n_tiles = n_tiles;
  }
  LIN_TRY(launch_adapters_tc(a, h->rpad, h->type == MOE_FP16, st));
  return MOE_OK;
}

extern "C" moe_status moe_adapters_get_device_error(moe_adapters* h, uint32_t* code) {
  if (!h || !code) return bad(MOE_ERR_INVALID_ARG, "the handle and code are required");
  *code = 0;
  if (h->device >= 0 && h->device != current_device())
    return bad(MOE_ERR_INVALID_ARG, "the handle's memory is on another device than the current one");
  LIN_TRY(cudaDeviceSynchronize());
  if (!h->err) return MOE_OK;
  LIN_TRY(cudaMemcpy(code, h->err, sizeof(uint32_t), cudaMemcpyDeviceToHost));
  LIN_TRY(cudaMemset(h->err, 0, sizeof(uint32_t)));
  LIN_TRY(cudaDeviceSynchronize());  // cleared before a later call, on any stream, sets a bit
  return *code ? bad(MOE_ERR_DEVICE, "device error bits are set") : MOE_OK;
}
