// Internal launch interface between the plan/ABI layer (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// Sets the thread's moe_last_error() message and returns s (api.cu).
moe_status fail_message(moe_status s, const char* msg);
// 2-D byte tensor [rows][inner] (row pitch ld bytes, a multiple of 16), box {128, box_rows}, 128-byte
// swizzle: 8-bit rows as a GEMM operand.  Bytes beyond the extents read as zero (api.cu).
moe_status make_map_f8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t ld, int box_rows);
// 2-D bf16 tensor [rows][inner] (row pitch ld elements, a multiple of 8), box {64, 32}, 128-byte swizzle.
moe_status make_map_bf16_out(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t ld);

// A conversion of x (bf16) that a kernel performs on the side with every thread of its grid: to x16
// (fp16, n8 * 8 elements; the 4-bit path's activation copy, convert_x16 in common.cuh), or to xq / xs
// (8-bit blocks of `rows` rows of K elements; the 8-bit path's operand, convert_x8 in fp8.cuh).
// Both nullptr: none.
struct XConv {
  const uint16_t* x = nullptr;
  uint16_t* x16 = nullptr;
  size_t n8 = 0;
  uint8_t* xq = nullptr;
  float* xs = nullptr;
  int rows = 0, K = 0;
  int64_t ldq = 0, lds = 0;
};

// Tokens per chunk of the grouping step: one 32-bit mask word per (chunk, expert).
constexpr int kChunk = 32;
// Row stride (32-bit words) of the per-chunk expert masks masks[e][c] for n_chunks chunks: a
// multiple of 4, so that rows are read as 16-byte vectors.
__host__ __device__ inline int group_mask_stride(int n_chunks) { return (n_chunks + 3) & ~3; }
// Largest number of rows one tensor-core unit handles (the MMA's N).
constexpr int kSegRowsMax = 128;

// One segment of the grouped problem: `rows` consecutive grouped rows of one expert starting
// at `row_start`.  An expert with more than kSegRowsMax rows has several parts; `first` is
// the index of its first part in the segment list, `nparts` their number, and `start` and `total`
// the expert's rows over all parts, so that one record locates every part.
struct Seg {
  int expert;
  int row_start;
  int rows;
  int first;
  int nparts;
  int start, total, pad;
};

// Scored selection (scored.cuh); on == 0: the softmax of the k largest logits.
constexpr int kMaxGroups = 32;  // a lane of the selecting warp holds a group's score
struct ScoreArgs {
  int on = 0;
  int sigmoid = 0;                // else softmax
  int groups = 1, keep = 1, top = 1;
  int renorm = 1;
  float scale = 1.0f;
  const float* bias = nullptr;    // [E] or NULL
  // lanes that share a group's members (a power of two, groups * lanes <= 32); ceil(2^20 / group size),
  // which divides an expert index exactly (index and size below 1024)
  int lanes = 1;
  uint32_t per_magic = 0;
};

// ---- routing and grouping (route.cu) --------------------------------------------------------
// logits[t][e] = x[t] . w_router[e] + b[e] (fp32 accumulation).
cudaError_t launch_router_logits(const uint16_t* x, const float* w_router, const float* b_router, int T,
                                 int E, int d, float* logits, cudaStream_t st);
// Top-k + softmax gates per token.  The logits are sum_s parts[s][T][E] (+ bias[e]) and are
// written to logits_out if given.  If masks != nullptr also writes the per-chunk expert masks,
// expert-major: bit t of masks[e * n_chunks + c] <=> token c*32+t chose e.
// xc: an x -> fp16 conversion the launch performs on the side (none by default).
cudaError_t launch_topk(const float* parts, int nsplit, const float* bias, float* logits_out, int T, int E, int k,
                        int32_t* ids, float* gates, uint32_t* masks, uint32_t* err, cudaStream_t st,
                        const XConv& xc = XConv{}, const ScoreArgs& sa = ScoreArgs{});

// ---- tensor-core router (router_tc.cu) --------------------------------------------------------
// parts[s][T][E] = x[T][k-range s] . W_r[E][k-range s]^T with W_r split into three bf16 pieces
// (w3: 2-D map over [3E rows][d], box 64 x 128).  Requires E % 128 == 0 and d % 64 == 0.
int router_tc_splits(int T, int E, int d, int num_sms);
constexpr int kRouterTcMinT = 16;  // the tensor-core router serves T > 16

// Small-T router (d % 128 == 0): K-split partials parts[router_small_splits(d)][T][E], no bias.
int router_small_splits(int d);
cudaError_t launch_router_parts_small(const uint16_t* x, const float* w_router, int T, int E, int d, float* parts,
                                      cudaStream_t st);

// Top-k + counts + offsets + segments + stable permutation of a small step in one launch.
constexpr int kSmallRouteT = 64;
bool route_small_ok(int T, int E, int k, int nsplit);
// Router + top-k + grouping of a step of at most 8 tokens (d % 128 == 0) in one launch.
bool router_route_tiny_ok(int T, int E, int d, int k);
cudaError_t launch_router_route_tiny(const uint16_t* x, const float* w_router, const float* bias, int T, int E, int d,
                                     float* parts, int k, int32_t* ids, float* gates, int32_t* counts,
                                     int32_t* offsets, int32_t* perm, int32_t* inv, Seg* segs, int32_t* n_segs,
                                     int max_segs, uint32_t* done, uint32_t* err, cudaStream_t st,
                                     const XConv& xc = XConv{}, const ScoreArgs& sa = ScoreArgs{});

// `done`: a device counter that is 0 between launches (the last block resets it).
cudaError_t launch_route_small(const float* parts, int nsplit, const float* bias, int T, int E, int k, int32_t* ids,
                               float* gates, int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, Seg* segs,
                               int32_t* n_segs, int max_segs, uint32_t* done, uint32_t* err, cudaStream_t st,
                               const XConv& xc = XConv{}, const ScoreArgs& sa = ScoreArgs{});
// Persistent: min(items, num_sms) CTAs over the (expert tile, K split, token tile) items.
// xm: x [T][d] bf16, box {64, 128}, 128-byte swizzle.
cudaError_t launch_router_tc(const CUtensorMap* w3, const CUtensorMap* xm, int T, int E, int d, int nsplit,
                             float* parts, uint32_t* err, int num_sms, cudaStream_t st);
cudaError_t launch_split_router(const float* w, uint16_t* w3, size_t n, cudaStream_t st);
// Per-chunk expert masks from given ids (validates range / duplicates).
// xc: 8-bit blocks of x, made on the side by blocks of their own.
cudaError_t launch_masks_from_ids(const int32_t* ids, int T, int E, int k, uint32_t* masks,
                                  uint32_t* err, cudaStream_t st, const XConv& xc = XConv{});
// Grouping of a small step (route_small_ok) from given ids in one launch: the masks and group
// launches' results, and xc as above.
cudaError_t launch_group_ids(const int32_t* ids, int T, int E, int k, int32_t* counts, int32_t* offsets, int32_t* perm,
                             int32_t* inv, Seg* segs, int32_t* n_segs, int max_segs, uint32_t* err, cudaStream_t st,
                             const XConv& xc = XConv{});
// Grouping in one launch from the chunk masks and the ids: counts, offsets (exclusive scan of
// counts, offsets[E] = total), perm / inv_perm (-1 for a dropped assignment) and, if segs is
// given, the segment list of the routed experts for the grouped GEMMs.
cudaError_t launch_group(const int32_t* ids, const uint32_t* masks, int T, int E, int k, int32_t* counts,
                         int32_t* offsets, int32_t* perm, int32_t* inv, Seg* segs, int32_t* n_segs, int max_segs,
                         uint32_t* err, cudaStream_t st);
// Segment list from offsets only (used by the separate experts entry point).
cudaError_t launch_segments_from_offsets(const int32_t* offsets, int E, Seg* segs, int32_t* n_segs,
                                         int max_segs, uint32_t* err, cudaStream_t st);

// ---- expert FFN, CUDA-core reference path (ffn_simt.cu) -------------------------------------
struct FfnWeights {
  // Routed experts.  bf16: w_gu [E][2f][d] with gate/up rows interleaved in groups of 8
  // (rows 16q..16q+7 = gate rows 8q..8q+7, rows 16q+8..16q+15 = up rows 8q..8q+7),
  // w_down [E][d][f] held as fp16.  MXFP4: the same row order for codes [.][.][K/2] and scales
  // [.][.][K/32]; w_down codes [E][d][f/2].
  const void* w_gu = nullptr;
  const uint8_t* s_gu = nullptr;
  const void* w_down = nullptr;
  const uint8_t* s_down = nullptr;
  int fp4 = 0;
  // Shared experts, n_shared concatenated: w_gu_s bf16 [n_s*2*f_s][d] interleaved the same
  // way per expert, w_down_s fp16 [n_s][d][f_s].
  const uint16_t* w_gu_s = nullptr;
  const uint16_t* w_down_s = nullptr;
  int n_shared = 0;
  int f_s = 0;
  int E = 0, k = 0, d = 0, f = 0;
  uint32_t* err = nullptr;
  // 1: bf16 routed / shared weights are in the tile-contiguous layouts of the tensor-core path;
  // fp4_tiled: 4-bit routed weights in the launch_tile_fp4 layout (scales inside the blocks)
  int tiled = 0, tiled_s = 0, fp4_tiled = 0;
};

// h, h_s, y, y_s are fp16.
cudaError_t launch_ffn_simt(const FfnWeights& w, const uint16_t* x, int T, const int32_t* offsets,
                            const int32_t* perm, uint16_t* h, uint16_t* h_s, uint16_t* y,
                            uint16_t* y_s, cudaStream_t st);

// ---- expert FFN, tcgen05 path (gemm_tc.cu) ---------------------------------------------------
struct TcMaps {
  CUtensorMap h;         // B for down: [R_max rows][f] fp16, box 64 x 32
  CUtensorMap h_s;       // B for shared down: [T_max rows][n_s*f_s] fp16, box 64 x 32
};

struct TcArgs {
  // tile-contiguous weights (launch_tile_gate_up / launch_tile_down layouts)
  const uint16_t* w_gu = nullptr;    // [E][f/64][d/64] blocks, bf16
  const uint16_t* w_gu_s = nullptr;  // [n_s*f_s/64][d/64] blocks, bf16
  const uint16_t* w_down = nullptr;  // [E][d/128][f/64] blocks, fp16
  const uint16_t* w_down_s = nullptr;  // [d/128][n_s][f_s/64] blocks, fp16
  // 4-bit routed weights (launch_tile_fp4 layout) for the fp4 kernels
  const uint8_t* q_gu = nullptr;     // [E][f/64][d/64] blocks of kFp4BlockBytes
  const uint8_t* q_down = nullptr;   // [E][d/128][f/64] blocks
  const uint16_t* x16 = nullptr;     // fp16 copy of x (4-bit path's B operand)
  const uint8_t* xq = nullptr;       // x as two e4m3 terms [T][2][d] (block-scaled gate/up's B operand)
  const uint8_t* xs = nullptr;       // their e8m0 scales [T][2][d / 32]
  uint32_t* sched = nullptr;         // persistent 4-bit kernels: the launch's unit hand-out words
  int routed = 1;                    // 0: the 16-bit kernels run the shared-expert units only
  const Seg* segs = nullptr;
  const int32_t* n_segs = nullptr;
  const int32_t* perm = nullptr;
  const uint16_t* x = nullptr;
  uint16_t* h = nullptr;
  uint16_t* h_s = nullptr;
  uint16_t* y = nullptr;
  uint16_t* y_s = nullptr;
  uint32_t* err = nullptr;
  int T = 0, E = 0, k = 0, d = 0, f = 0, n_shared = 0, f_s = 0;
  int n_shared_segs = 0;   // ceil(T / kSegRowsMax) when n_shared > 0 (shared tokens split evenly)
  int pair = 2;            // bf16 kernels: weight tiles per unit (2 shares each B stage; 1 for few units)
};

cudaError_t launch_tc_gateup(const TcMaps* maps, const TcArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_tc_down(const TcMaps* maps, const TcArgs& a, int num_sms, cudaStream_t st);

// ---- expert FFN with 4-bit routed weights, tcgen05 (gemm_fp4.cu) -----------------------------
// Routed units only (shared experts go through the 16-bit kernels with routed = 0).
cudaError_t launch_fp4_gateup(const TcMaps* maps, const TcArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_fp4_down(const TcMaps* maps, const TcArgs& a, int num_sms, cudaStream_t st);
// x16 = fp16(x), n elements (multiple of 8); out-of-range values clamp and flag MOE_DEVERR_RANGE.
cudaError_t launch_x_to_f16(const uint16_t* x, uint16_t* x16, size_t n, uint32_t* err, cudaStream_t st);
// ---- 4-bit gate/up on the block-scaled MMA (gemm_mx.cu) ------------------------------------------
// xq [T][2][d] e4m3 (hi, lo) and xs [T][2][d / 32] e8m0 from x (bf16); requires d % 128 == 0.
cudaError_t launch_x_to_mx(const uint16_t* x, uint8_t* xq, uint8_t* xs, int T, int d, cudaStream_t st);
// h = SwiGLU of the routed units (a.q_gu tiled 4-bit weights, a.xq / a.xs, a.sched: zeroed words
// [0] units handed out, [1] CTAs exited; the last CTA resets them).
cudaError_t launch_mx_gateup(const TcArgs& a, int num_sms, cudaStream_t st);
// y (fp16) of the routed units from W_down (a.q_down) and h in two e4m3 terms: a.xq = hq
// [R][2][f], a.xs = hs [R][2][mx_scale_bytes(f)] (launch_h_to_mx), a.sched as above.
cudaError_t launch_mx_down(const TcArgs& a, int num_sms, cudaStream_t st);
// hq / hs from h (fp16 [R][f]); f % 64 == 0.
cudaError_t launch_h_to_mx(const uint16_t* h, uint8_t* hq, uint8_t* hs, int R, int f, cudaStream_t st);
// scale bytes per quantised row of K elements (K / 32 rounded up to a multiple of 4)
int mx_scale_bytes(int K);

// ---- 8-bit block-scaled path (quant_fp8.cu, gemm_fp8.cu) ---------------------------------------
// One stage tile of 8-bit weights: 128 rows x 128 K elements, stored as the 128-byte-swizzled K-major
// shared-memory image ((r, 16-byte chunk c) at r * 128 + ((c ^ (r & 7)) << 4)).  A GEMM tile is 256
// weight rows, two such halves, adjacent at each K block (a lone last half stands alone):
//   linear / down: half h = rows 128 h .. 128 h + 127 of the matrix;
//   gate/up: half h = gate rows 64 h .. 64 h + 63, then the up rows of the same features; always
//     whole tiles (128 features, the block that shares one activation scale of h).
// Scales [matrix][tile][K block, padded to four][2]: the two 128-row blocks', or gate's and up's.
constexpr int kF8TileBytes = 128 * 128;
__host__ __device__ inline int f8_halves(int rows, bool gate_up) {
  return gate_up ? 2 * ((rows + 127) / 128) : (rows + 127) / 128;
}
__host__ __device__ inline int64_t f8_half_offset(int h, int kb, int halves, int nk) {
  const int t = h >> 1, np = halves - 2 * t < 2 ? 1 : 2;
  return (static_cast<int64_t>(t) * 2 * nk + static_cast<int64_t>(kb) * np + (h & 1)) * kF8TileBytes;
}
// Row pitch of an activation's block scales: 16-byte groups of four K blocks.
__host__ __device__ inline int f8_scale_ld(int nk) { return (nk + 3) & ~3; }

cudaError_t launch_quant_rows(const void* x, moe_dtype dt, int64_t ldx, int rows, int K, uint8_t* q, int64_t ldq,
                              float* s, int64_t lds, int num_sms, cudaStream_t st);
cudaError_t launch_quant_blocks(const void* w, moe_dtype dt, int64_t ldw, int rows, int K, uint8_t* q, int64_t ldq,
                                float* s, int64_t lds, cudaStream_t st);
// n matrices [rows][K] of codes (b != nullptr: gate = a and up = b) and their scales
// [n][ceil(rows/128)][ceil(K/128)] into the layout above.
cudaError_t launch_tile_fp8(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb, uint8_t* dst,
                            float* sdst, int n, int rows, int K, cudaStream_t st);

struct F8Args {
  const uint8_t* w = nullptr;   // tiled weights; matrix stride w_stride bytes
  const float* ws = nullptr;    // tiled scales
  int64_t w_stride = 0;
  const uint8_t* a = nullptr;   // gate/up: e4m3 rows of x (gathered by perm), pitch lda bytes
  int64_t lda = 0;
  const float* as = nullptr;    // activation scales, pitch lds floats (a multiple of 4)
  int64_t lds = 0;
  const Seg* segs = nullptr;    // routed rows; linear: the T rows split evenly
  const int32_t* n_segs = nullptr;
  const int32_t* perm = nullptr;
  uint8_t* hq = nullptr;        // gate/up out: e4m3 rows [grouped rows][ldh], scales [.][ldhs]
  float* hs = nullptr;
  int64_t ldh = 0, ldhs = 0;
  void* out = nullptr;          // linear / down out [rows][ldo] of out_type, columns < N
  int64_t ldo = 0;
  int out_type = MOE_FP16;      // fp16 (the layer's y: clamped, flags MOE_DEVERR_RANGE), bf16 or fp32
  int out_vec = 0;              // rows start, and N ends, on 16-byte boundaries
  int N = 0, halves = 0, nk = 0;
  int T = 0, k = 0;
  int box_rows = 32;            // rows of amap's box (a multiple of 32)
  int splits = 1;               // linear: CTAs of a cluster that share a unit's K blocks (set at launch)
  uint32_t* err = nullptr;
};
// amap: the activation rows [rows][K] as bytes, box {128, a.box_rows}, 128-byte swizzle (not gate/up);
// amap128: the same with 128 rows.
cudaError_t launch_f8_gateup(const F8Args& a, int num_sms, cudaStream_t st);
cudaError_t launch_f8_down(const CUtensorMap* amap, const CUtensorMap* amap128, const F8Args& a, int num_sms,
                           cudaStream_t st);
// omap: bf16 out with a.out_vec, [T][N], box {64, 32}, 128-byte swizzle (else unused).
cudaError_t launch_f8_linear(const CUtensorMap* amap, const CUtensorMap* omap, const F8Args& a, int num_sms,
                             cudaStream_t st);

// ---- one-launch layer of a small step (layer_small.cu) ------------------------------------------
constexpr int kLsTMax = 8;                  // tokens per step
constexpr int kLsUnionBytes = 76 * 1024;    // x (bf16) and then h (fp16) of the step in shared memory
constexpr int kLsSyncWords = 8;            // launch-wide counters and flags
struct LsArgs {
  const uint16_t* x = nullptr;
  const float* w_router = nullptr;
  const float* b_router = nullptr;
  const uint16_t* w_gu = nullptr;      // tile-contiguous layouts of the tensor-core path
  const uint16_t* w_down = nullptr;
  const uint16_t* w_gu_s = nullptr;
  const uint16_t* w_down_s = nullptr;
  float* logits = nullptr;             // [T][E]
  int32_t* ids = nullptr;              // [T][k]
  float* gates = nullptr;              // [T][k]
  int32_t* counts = nullptr;           // [E]
  int32_t* offsets = nullptr;          // [E + 1]
  int32_t* perm = nullptr;             // [T k]
  int32_t* inv = nullptr;              // [T k]
  int32_t* touched = nullptr;          // [E]: touched experts, ascending
  int32_t* n_touched = nullptr;        // 1 word
  uint16_t* h = nullptr;               // fp16 [T k][f] grouped rows
  uint16_t* h_s = nullptr;             // fp16 [T][n_s f_s]
  float* y32 = nullptr;                // fp32 [T k][d] per assignment t k + j
  float* ys32 = nullptr;               // fp32 [T][d]
  uint16_t* out = nullptr;             // bf16 [T][d]
  uint32_t* sync = nullptr;            // kLsSyncWords plan-owned words, zero between launches
  uint32_t* err = nullptr;
  int T = 0, E = 0, k = 0, d = 0, f = 0, n_shared = 0, f_s = 0;
};
bool layer_small_ok(int T, int E, int k, int d, int f, int n_shared, int f_s);
cudaError_t launch_layer_small(const LsArgs& a, int num_sms, cudaStream_t st);

// ---- combine (combine.cu): out bf16; y and shared_y fp16 (the layer's intermediates) or fp32 ----
cudaError_t launch_combine(const uint16_t* y, const float* gates, const int32_t* inv,
                           const uint16_t* shared_y, int T, int k, int d, uint16_t* out,
                           cudaStream_t st);
cudaError_t launch_combine_f32(const float* y, const float* gates, const int32_t* inv, const float* shared_y, int T,
                               int k, int d, uint16_t* out, cudaStream_t st);

// ---- weight repacking at set-up (repack.cu) --------------------------------------------------
// dst [n][2f][K*elem] <- gate [n][f][K*elem], up [n][f][K*elem], rows interleaved by 8.
cudaError_t launch_interleave_gate_up(const uint8_t* gate, const uint8_t* up, uint8_t* dst, int n,
                                      int f, size_t row_bytes, cudaStream_t st);
// dst fp16 <- src bf16 (round to nearest even); *bad |= 1 if a value is outside the fp16 range.
cudaError_t launch_bf16_to_f16(const uint16_t* src, uint16_t* dst, size_t n, uint32_t* bad, cudaStream_t st);
// Tile-contiguous, pre-swizzled layouts of the tensor-core path (16 KB blocks of 128 rows x 64
// K elements).  A weight matrix of `tiles` 128-row tiles and nk K chunks stores its blocks at
// tile_chunk_offset: tiles are paired and the two tiles of a pair alternate along K, so both
// blocks of one K chunk are adjacent (one 32 KB copy); an odd last tile stands alone.
//   gate/up of n experts (rows interleaved by 8): one matrix per expert (f/64 tiles, d/64 chunks),
//     or with one_matrix the n experts as one matrix of n f/64 tiles (the shared experts);
//   down (bf16 -> fp16) of n matrices [rows][K]: by_matrix ? one matrix per expert (rows/128
//     tiles, K/64 chunks) : one matrix of rows/128 tiles whose K runs over all n (n K/64 chunks).
cudaError_t launch_tile_gate_up(const uint16_t* gate, const uint16_t* up, uint16_t* dst, int n, int f, int d,
                                int one_matrix, cudaStream_t st);
cudaError_t launch_tile_down(const uint16_t* src, uint16_t* dst, int n, int rows, int K, int by_matrix, uint32_t* bad,
                             cudaStream_t st);
constexpr int kTileElems = 128 * 64;
// 4-bit tile-contiguous blocks (launch_tile_fp4): 128 rows x 64 K elements, codes then scales.
constexpr int kFp4BlockBytes = 4096 + 256;
// e8m0 scale bytes for which e2m1 x 2^(s-127) is exact in fp16 (subnormals included): the
// tensor-core 4-bit path dequantises into fp16.
constexpr int kFp4ScaleMin = 104;
constexpr int kFp4ScaleMax = 140;
cudaError_t launch_tile_fp4(const uint8_t* codes_a, const uint8_t* scales_a, const uint8_t* codes_b,
                            const uint8_t* scales_b, uint8_t* dst, int n, int rows, int K, int gate_up,
                            uint32_t* scale_oor, cudaStream_t st);
// Element offset of block (tile t, K chunk kc) inside one tile-contiguous weight matrix.
__host__ __device__ inline size_t tile_chunk_offset(int t, int kc, int tiles, int nk) {
  const int pr = t >> 1, w = t & 1;
  const int np = tiles - 2 * pr < 2 ? tiles - 2 * pr : 2;
  return (static_cast<size_t>(pr) * 2 * nk + static_cast<size_t>(kc) * np + w) * kTileElems;
}
// Elements between consecutive K chunks of tile t (2 blocks inside a pair, 1 for a lone tile).
__host__ __device__ inline size_t tile_chunk_stride(int t, int tiles) {
  return static_cast<size_t>(tiles - 2 * (t >> 1) < 2 ? 1 : 2) * kTileElems;
}
// Element offset of (row r, K element kk) inside one 128 x 64 block (128-byte swizzle).
__host__ __device__ inline size_t tile_elem_offset(int r, int kk) {
  return static_cast<size_t>(r) * 64 + ((((kk >> 3) ^ (r & 7)) << 3) | (kk & 7));
}

}  // namespace moe
