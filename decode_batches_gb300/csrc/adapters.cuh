// Low-rank adapters: interface between the C entry points (adapters_api.cu) and the kernels (adapters.cu).
#pragma once

#include "kernels.h"

namespace moe {

constexpr int kAdaptersMax = 1024;    // slots of a handle
constexpr int kAdapterRankMax = 128;
constexpr int kAdapterScan = 256;     // rows up to which a cluster finds its tile itself
constexpr int kAdapterCount = 1024;   // rows up to which the larger steps' clusters count the ids themselves
constexpr int kAdapterTileRows = 128; // rows of a grouped tile at most

// Rows [start, start + rows) of `order` that share a slot (slot -1: rows without an adapter), with what a tile needs to
// know of it.
struct alignas(16) AdapterTile {
  int slot, start;
  uint16_t rows, rank;
  float scale;
};
struct AdapterSlots {
  const int32_t* rank = nullptr;    // [n] ranks, 0: empty slot
  const float* scale = nullptr;     // [n]
};
// How a step of T rows is cut: rows of a tile at most, CTAs that share a tile.
struct AdapterCut {
  int rows = 128, ctas = 1;
  int slots = 1;                    // CTAs that run at a time
  bool small = false;               // two CTAs of 8 warps an SM, else one of 16
};
// A slot's `all` rows are cut evenly, in multiples of 16: rows of each of its tiles but the last.
__host__ __device__ inline int adapter_tile_rows(int all, int most) {
  const int parts = (all + most - 1) / most;
  return ((all + parts - 1) / parts + 15) / 16 * 16;
}
AdapterCut adapter_cut(int T, int n, int rpad, int num_sms);
int adapter_clusters(int T, int n, const AdapterCut& cut, bool copies);

struct AdapterArgs {
  const uint16_t* x = nullptr;      // [T][K]
  int64_t ldx = 0;
  const int32_t* ids = nullptr;     // [T]
  const uint16_t* a = nullptr;      // packed A of all slots (adapter_pack)
  const uint16_t* b = nullptr;      // packed B
  const uint16_t* a_tc = nullptr;   // the same as the tensor cores' operand tiles (adapter_tc_pack)
  const uint16_t* b_tc = nullptr;
  int64_t a_tc_slot = 0, b_tc_slot = 0;
  AdapterSlots slots;
  const void* base = nullptr;       // [T][N] of out_type, or NULL (zero)
  int64_t ld_base = 0;
  void* out = nullptr;
  int64_t ld_out = 0;
  int out_type = MOE_BF16;
  int x_vec = 0, out_vec = 0;       // rows of x / of base and out are 16-byte aligned, K / N a multiple of 8
  int T = 0, n = 0, K = 0, N = 0;
  AdapterCut cut;                   // (the small steps' is set at launch)
  int64_t a_slot = 0, b_slot = 0;   // elements of a slot's packed A, B
  const int32_t* order = nullptr;   // grouped rows and their tiles (larger T)
  const AdapterTile* tiles = nullptr;
  const int32_t* n_tiles = nullptr;
  uint32_t* err = nullptr;
};

inline int adapter_rank_pad(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }
inline int64_t adapter_a_elems(int K, int rpad) { return static_cast<int64_t>((K + 31) / 32) * 32 * rpad; }
inline int64_t adapter_b_elems(int N, int rpad) { return static_cast<int64_t>((N + 31) / 32) * 32 * rpad; }

inline int64_t adapter_tc_a_elems(int K, int rpad) { return static_cast<int64_t>((K + 63) / 64) * 64 * rpad; }
inline int64_t adapter_tc_b_elems(int N, int rpad) { return static_cast<int64_t>((N + 127) / 128) * 128 * rpad; }

// One slot's A [r][K] and B [N][r] into the kernels' order.
cudaError_t launch_adapter_pack(const uint16_t* a, const uint16_t* b, uint16_t* pa, uint16_t* pb, int r, int K, int N,
                                int rpad, cudaStream_t st);
cudaError_t launch_adapter_tc_pack(const uint16_t* a, const uint16_t* b, uint16_t* pa, uint16_t* pb, int r, int K, int N,
                                   int rpad, cudaStream_t st);
// order [T] (the rows without an adapter last), tiles, and n_tiles: their number, the place of the first row without an
// adapter, the rows of a tile at most, n_tiles from ids; ids outside [-1, n) set MOE_DEVERR_EXPERT_RANGE.
cudaError_t launch_adapter_group(const int32_t* ids, int T, int n, const AdapterCut& cut, const AdapterSlots& slots,
                                 int32_t* order, AdapterTile* tiles, int32_t* n_tiles, uint32_t* err, cudaStream_t st);
cudaError_t launch_adapters(const AdapterArgs& p, int rpad, bool fp16, int num_sms,
                            cudaStream_t st);                        // T <= kAdapterScan
cudaError_t launch_adapters_tc(const AdapterArgs& p, int rpad, bool fp16, cudaStream_t st);  // p.tiles: T > kAdapterCount

}  // namespace moe
