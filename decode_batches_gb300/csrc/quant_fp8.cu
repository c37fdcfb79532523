// Quantisation into e4m3 blocks, and the set-up repacking of 8-bit weights.
//
// quant_rows: rows [T][K] (bf16, fp16 or fp32, any row pitch) -> codes [T][ldq] and one fp32 scale
//   per 128 elements of a row, in one pass (quant_rows_part).  Bound by memory: K (2 + 1) bytes a
//   bf16 row.
// quant_blocks: a matrix [rows][K] -> codes and one scale per 128 x 128 block (weights; set-up).
// tile_fp8: codes [n][rows][K] into the tile-contiguous, pre-swizzled layout of the 8-bit GEMMs.
#include "fp8.cuh"
#include "kernels.h"

namespace moe {

constexpr int kQuantThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 4 : 2) quant_rows_kernel(const T* __restrict__ x, int64_t ldx, int rows, int K,
                                                                   int nb, int vec, uint8_t* __restrict__ q,
                                                                   int64_t ldq, float* __restrict__ s, int64_t lds) {
  pdl_trigger();
  pdl_wait();
  quant_rows_part(x, ldx, rows, K, nb, vec != 0, q, ldq, s, lds, blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5),
                  gridDim.x * (kQuantThreads / 32));
}

static bool vec_ok(const void* p, int64_t ld, size_t elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (static_cast<size_t>(ld) * elem) % 16 == 0;
}

template <typename T>
static cudaError_t launch_quant_rows_t(const void* x, int64_t ldx, int rows, int K, uint8_t* q, int64_t ldq, float* s,
                                       int64_t lds, int num_sms, cudaStream_t st) {
  const int nb = (K + kF8Block - 1) / kF8Block;
  const int64_t warps = static_cast<int64_t>(rows) * ((nb + 7) / 8);
  const int64_t blocks = (warps + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
  const int64_t most = static_cast<int64_t>(num_sms) * 4;  // the resident blocks
  return launch_pdl(quant_rows_kernel<T>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                    dim3(kQuantThreads), 0, st, static_cast<const T*>(x), ldx, rows, K, nb,
                    vec_ok(x, ldx, sizeof(T)) ? 1 : 0, q, ldq, s, lds);
}

cudaError_t launch_quant_rows(const void* x, moe_dtype dt, int64_t ldx, int rows, int K, uint8_t* q, int64_t ldq,
                              float* s, int64_t lds, int num_sms, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  if (dt == MOE_BF16) return launch_quant_rows_t<__nv_bfloat16>(x, ldx, rows, K, q, ldq, s, lds, num_sms, st);
  if (dt == MOE_FP16) return launch_quant_rows_t<__half>(x, ldx, rows, K, q, ldq, s, lds, num_sms, st);
  return launch_quant_rows_t<float>(x, ldx, rows, K, q, ldq, s, lds, num_sms, st);
}

// ---- weights: 128 x 128 blocks ---------------------------------------------------------------
MOE_DEVICE float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
MOE_DEVICE float to_f32(__half v) { return __half2float(v); }
MOE_DEVICE float to_f32(float v) { return v; }

template <typename T>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const T* __restrict__ w, int64_t ldw, int rows, int K,
                                                           uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ s,
                                                           int64_t lds) {
  __shared__ float part[8];
  const int k = blockIdx.x * kF8Block + (threadIdx.x & 127);
  const int r0 = blockIdx.y * kF8Block + (threadIdx.x >> 7);  // rows r0, r0 + 2, ...
  float v[64], amax = 0.f;
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const int r = r0 + 2 * i;
    v[i] = (r < rows && k < K) ? to_f32(w[r * ldw + k]) : 0.f;
    amax = fmaxf(amax, fabsf(v[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, part[i]);
  const float sc = f8_scale(amax);
  const float r = __frcp_rn(sc);
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const int rr = r0 + 2 * i;
    if (rr < rows && k < K) q[rr * ldq + k] = static_cast<uint8_t>(f32x2_to_e4m3x2(v[i] * r, 0.f));
  }
  if (threadIdx.x == 0) s[blockIdx.y * lds + blockIdx.x] = sc;
}

cudaError_t launch_quant_blocks(const void* w, moe_dtype dt, int64_t ldw, int rows, int K, uint8_t* q, int64_t ldq,
                                float* s, int64_t lds, cudaStream_t st) {
  const dim3 grid((K + kF8Block - 1) / kF8Block, (rows + kF8Block - 1) / kF8Block);
  if (dt == MOE_BF16)
    quant_blocks_kernel<<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(w), ldw, rows, K, q, ldq, s, lds);
  else if (dt == MOE_FP16)
    quant_blocks_kernel<<<grid, 256, 0, st>>>(static_cast<const __half*>(w), ldw, rows, K, q, ldq, s, lds);
  else
    quant_blocks_kernel<<<grid, 256, 0, st>>>(static_cast<const float*>(w), ldw, rows, K, q, ldq, s, lds);
  return cudaGetLastError();
}

// ---- weights into the GEMM's layout ------------------------------------------------------------
// One thread moves one 16-byte chunk of the destination: [matrix][tile][K block][half][128 rows][128]
// (a lone last half has no partner).  Rows and columns beyond the matrix become zero codes.
__global__ void __launch_bounds__(256) tile_fp8_kernel(const uint8_t* __restrict__ a, const uint8_t* __restrict__ b,
                                                       uint8_t* __restrict__ dst, int rows, int K, int halves, int nk,
                                                       int64_t chunks, int vec) {
  const int64_t per = static_cast<int64_t>(halves) * nk * (kF8TileBytes / 16);  // chunks of one matrix
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < chunks; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t m = i / per;
    int64_t o = i - m * per;                   // half-tile order (half, kb) first, decoded to find its place
    const int c = static_cast<int>(o & 7);     // logical 16-byte chunk of the row
    const int r = static_cast<int>((o >> 3) & 127);
    o >>= 10;
    const int kb = static_cast<int>(o % nk), h = static_cast<int>(o / nk);
    const uint8_t* src;
    int row;
    if (b) {  // gate/up: half h = 64 gate rows, then the same 64 features' up rows
      src = r < 64 ? a : b;
      row = 64 * h + (r & 63);
    } else {
      src = a;
      row = 128 * h + r;
    }
    const int k = kb * kF8Block + 16 * c;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (row < rows && k < K) {
      const uint8_t* p = src + (m * rows + row) * static_cast<int64_t>(K) + k;
      if (vec) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else {
        for (int j = 0; j < 16; ++j)
          if (k + j < K) w[j >> 2] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
      }
    }
    uint8_t* d = dst + m * per * 16 + f8_half_offset(h, kb, halves, nk) + r * 128 + ((c ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Scales [n][rb][nk] (one matrix, or gate and up) -> [n][tiles][f8_scale_ld(nk)][2].
__global__ void __launch_bounds__(256) tile_scales_kernel(const float* __restrict__ a, const float* __restrict__ b,
                                                          float* __restrict__ dst, int n, int rb, int tiles, int nk) {
  const int ld = f8_scale_ld(nk);
  const int64_t total = static_cast<int64_t>(n) * tiles * ld * 2;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int w = static_cast<int>(i & 1);
    const int64_t o = i >> 1;
    const int kb = static_cast<int>(o % ld);
    const int t = static_cast<int>((o / ld) % tiles);
    const int64_t m = o / ld / tiles;
    const int blk = b ? t : 2 * t + w;
    const float* src = (b && w) ? b : a;
    dst[i] = blk < rb && kb < nk ? src[(m * rb + blk) * nk + kb] : 0.f;
  }
}

cudaError_t launch_tile_fp8(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb, uint8_t* dst,
                            float* sdst, int n, int rows, int K, cudaStream_t st) {
  const int halves = f8_halves(rows, b != nullptr), nk = (K + kF8Block - 1) / kF8Block;
  const int tiles = (halves + 1) / 2, rb = (rows + kF8Block - 1) / kF8Block;
  const int64_t chunks = static_cast<int64_t>(n) * halves * nk * (kF8TileBytes / 16);
  const int64_t blocks = (chunks + 255) / 256;
  const int vec = K % 16 == 0 && (reinterpret_cast<uintptr_t>(a) & 15) == 0 && (reinterpret_cast<uintptr_t>(b) & 15) == 0;
  tile_fp8_kernel<<<static_cast<unsigned>(blocks < 65536 ? blocks : 65536), 256, 0, st>>>(a, b, dst, rows, K, halves, nk,
                                                                                         chunks, vec);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t ns = static_cast<int64_t>(n) * tiles * f8_scale_ld(nk) * 2;
  tile_scales_kernel<<<static_cast<unsigned>((ns + 255) / 256 < 4096 ? (ns + 255) / 256 : 4096), 256, 0, st>>>(sa, sb, sdst, n,
                                                                                                    rb, tiles, nk);
  return cudaGetLastError();
}

}  // namespace moe
