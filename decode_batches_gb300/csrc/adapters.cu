// Low-rank adapters of many requests (include/moe.h: moe_adapters_forward):
//   out[t] = base[t] + B_a (s_a A_a x[t]),  a = ids[t].
//
// A tile is up to M rows of one adapter; a cluster of CTAs computes it in one pass: each warp multiplies its
// own range of K (shrink), the partial sums of u = A x meet in shared memory and then over the cluster, every
// CTA holds the whole u, and each warp multiplies its own range of the features (expand), adds the base and
// writes.  So x, base and the weights are read once and u never leaves the chip.
//
// This file has the steps of at most 256 rows (and the grouping of larger ones, which run in adapters_tc.cu).  Such a
// step streams its adapters' weights once, a few rows a tile, so the products run on warp-level fragments and no
// operand is shared between warps: the weights are packed in fragment order, and the k index of the shrink (any order
// will do) is dealt to the lanes such that a lane's share of a row is 16 contiguous bytes.  The expand's features are
// dealt so that a lane's results are eight neighbours of a row.  Bound by latency: ids, rank, weights, two cluster
// barriers, 4.8 us for one row (rank 16, 4096 x 4096) of which a launch is 2; 48 rows of 35 adapters of rank 64 16.5 us,
// 2.2 TB/s of weights.
//
// u is split in 16-bit terms, three in bf16 (all of its 24 bits; a 16-bit result takes the first two, 2^-16 of u) and
// two in fp16 (22 bits), since one term's 2^-8 would dominate the result.  In fp16 a row's u is first brought to the upper
// end of the type's range by a power of two, so that neither term leaves it.
#include "adapters.cuh"
#include "adapters_split.cuh"
#include "cluster.cuh"
#include "elems.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTileRows = 16;

template <bool kFp16>
MOE_DEVICE void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (kFp16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory of a CTA.  Each warp has a ring of stages that its loads go through (cp.async): a stage holds a
// chunk of 32 columns of x and of A, or a chunk of 32 features of B.  A lane reads back exactly what it copied, so
// the ring needs no barrier.  The first stage of all warps also holds the shrink's partial sums.
template <int M, int R, bool kFp16>
struct Smem {
  static constexpr int kTerms = kAdapterTerms<kFp16>;
  static constexpr int kStageBytes = (M + R) * 64;
  static constexpr int kStages = kStageBytes <= 3072 ? 4 : 2;  // (two CTAs fit an SM up to rank 64)
  static constexpr int kPitch = R + (R % 32 == 0 ? 16 : 0);  // 16-bit elements: rows 8 apart share no bank
  static constexpr int kSlots = kWarps / 2;                  // partial sums are joined in pairs first
  union {
    uint8_t ring[kStages][kWarps][kStageBytes];
    struct {
      float warp_part[kSlots][M][R];
      float part[M][R];
    };
  };
  alignas(16) uint16_t u[kTerms][M][kPitch];
  float row_scale[M];                    // (fp16) the power of two that a row's u was divided by
  int rows[M];                           // the tile's rows, -1 past the last
  alignas(16) int ids[kThreads];
  uint32_t leads[kWarps];
  int tile[4];                           // slot, number of its first row, rank, is there one
  static_assert(kAdapterScan <= kThreads, "a thread a row");
  static_assert((kSlots + 1) * M * R * 4 <= kWarps * kStageBytes, "the partial sums fit one stage");
};

// The tile of the cluster, found in ids by every CTA for itself (a step has 256 rows at most): a row whose number among
// the rows of its id is a multiple of M leads a tile, and cluster i takes the i-th leader's, whose rows go to s.rows.
// Returns whether there is one, with its slot (-1: no adapter) and rank.  The same for every thread of the cluster.
template <int M, int R, bool kFp16>
MOE_DEVICE bool find_tile(const AdapterArgs& p, Smem<M, R, kFp16>& s, int& slot, int& rank) {
  const int idx = blockIdx.x / p.cut.ctas, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int id = -2;
  if (t < p.T) {
    id = p.ids[t];
    if (id < -1 || id >= p.n) {
      if (blockIdx.x == 0) set_error(p.err, MOE_DEVERR_EXPERT_RANGE);
      id = -1;
    }
  }
  const int own_rank = id >= 0 ? p.slots.rank[id] : 0;
  if (p.T <= 32) {  // one warp's ids: the first warp finds the tile without a barrier (1 us of 6 less for one row)
    if (warp == 0) {
      const uint32_t same = __match_any_sync(0xffffffffu, id);
      const int before = __popc(same & ((1u << lane) - 1u));
      const bool lead = t < p.T && before % M == 0;
      const uint32_t leads = __ballot_sync(0xffffffffu, lead);
      if (lane == 0) s.tile[3] = idx < __popc(leads);
      if (lead && __popc(leads & ((1u << lane) - 1u)) == idx) {
        s.tile[0] = id, s.tile[2] = own_rank;
        uint32_t left = same & ~((1u << lane) - 1u);  // the tile's rows: the leader's and the next M - 1 of its id
#pragma unroll
        for (int i = 0; i < M; ++i) s.rows[i] = left ? __ffs(left) - 1 : -1, left &= left - 1;
      }
    }
    __syncthreads();
    slot = s.tile[0], rank = s.tile[2];
    return s.tile[3];
  }
  if (t < M) s.rows[t] = -1;
  s.ids[t] = id;
  __syncthreads();
  int before = __popc(__match_any_sync(0xffffffffu, id) & ((1u << lane) - 1u));  // earlier rows of this id
  for (int i = 0; i < 32 * warp; i += 4) {
    const int4 v = *reinterpret_cast<const int4*>(&s.ids[i]);
    before += (v.x == id) + (v.y == id) + (v.z == id) + (v.w == id);
  }
  const bool lead = t < p.T && before % M == 0;
  const uint32_t leads = __ballot_sync(0xffffffffu, lead);
  if (lane == 0) s.leads[warp] = leads;
  __syncthreads();
  int number = __popc(leads & ((1u << lane) - 1u)), all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) number += all;
    all += __popc(s.leads[w]);
  }
  if (idx >= all) return false;
  if (lead && number == idx) s.tile[0] = id, s.tile[1] = before, s.tile[2] = own_rank;
  __syncthreads();
  slot = s.tile[0], rank = s.tile[2];
  const int at = before - s.tile[1];
  if (t < p.T && id == slot && at >= 0 && at < M) s.rows[at] = t;
  __syncthreads();
  return true;
}

// One chunk of 32 columns of the tile's rows and of A into a stage: x pieces (row 16 m + 8 h + g, columns 8 q ..)
// at ((2 m + h) * 32 + lane) * 16, A's fragments of 8 ranks j behind them.
template <int M, int R>
MOE_DEVICE void stage_shrink(const AdapterArgs& p, uint8_t* st, const uint16_t* const (&x_row)[M / 16][2], const uint4* wa,
                             int k, int nt, int lane) {
  const int col = 32 * k + 8 * (lane & 3);
  uint4* x = reinterpret_cast<uint4*>(st) + lane;
  if (p.x_vec && 32 * k + 32 <= p.K) {
#pragma unroll
    for (int i = 0; i < M / 8; ++i) cp_async_16(smem_u32(x + i * 32), x_row[i / 2][i % 2] + 32 * k);
  } else if (p.x_vec) {
#pragma unroll
    for (int i = 0; i < M / 8; ++i)
      cp_async_16_part(smem_u32(x + i * 32), col < p.K ? x_row[i / 2][i % 2] + 32 * k : p.x, col < p.K ? 16u : 0u);
  } else {
    for (int i = 0; i < M / 8; ++i) x[i * 32] = load_x(x_row[i / 2][i % 2] - 8 * (lane & 3), col, p.K);
  }
#pragma unroll
  for (int j = 0; j < R / 8; ++j)
    if (j < nt) cp_async_16(smem_u32(x + (M / 8 + j) * 32), wa + (static_cast<int64_t>(k) * (R / 8) + j) * 32);
}

// One chunk of 32 features of B into a stage.
template <int R>
MOE_DEVICE void stage_expand(uint8_t* st, const uint4* wb, int c, int rs, int lane) {
  uint4* w = reinterpret_cast<uint4*>(st) + lane;
#pragma unroll
  for (int k = 0; k < R / 8; ++k)
    if (k < 2 * rs) cp_async_16(smem_u32(w + k * 32), wb + (static_cast<int64_t>(c) * (R / 8) + k) * 32);
}

// The expand's loop over the warp's chunks of features.  The first kStages - 1 chunks are on their way already, in
// the stages from 1 on; u's fragments stay in registers where there
// are few, the base's rows are requested before the products.  Rank 0: the base as it is.
template <typename E, int M, int R, bool kFp16>
MOE_DEVICE void expand(const AdapterArgs& p, Smem<M, R, kFp16>& s, const uint4* wb, int c0, int c1, int rank, int lane, int warp) {
  constexpr int MT = M / 16, RS = R / 16, kStages = Smem<M, R, kFp16>::kStages;
  constexpr int kTerms = sizeof(E) == 4 ? kAdapterTerms<kFp16> : 2;  // (of a 16-bit result: below its own rounding)
  const int g = lane >> 2, q = lane & 3, rs = (rank + 15) / 16;
  const E* base[MT][2];
  E* out[MT][2];
  float mul[MT][2];
  uint32_t live = 0;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = s.rows[16 * m + g + 8 * h];
      if (r >= 0) live |= 1u << (2 * m + h);
      base[m][h] = p.base ? static_cast<const E*>(p.base) + max(r, 0) * p.ld_base + 8 * q : nullptr;
      out[m][h] = static_cast<E*>(p.out) + max(r, 0) * p.ld_out + 8 * q;
      mul[m][h] = kFp16 && rank > 0 ? s.row_scale[16 * m + g + 8 * h] : 1.0f;
    }
  constexpr bool kHold = MT * RS <= 4;
  uint2 u[kHold ? MT : 1][kHold ? RS : 1][kTerms][2];  // [.][.][term][row g, row g + 8]
#pragma unroll
  for (int m = 0; m < (kHold ? MT : 0); ++m)
#pragma unroll
    for (int k = 0; k < RS; ++k)
#pragma unroll
      for (int t = 0; t < kTerms; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          u[m][k][t][h] = *reinterpret_cast<const uint2*>(&s.u[t][16 * m + g + 8 * h][16 * k + 4 * q]);
  int slot = 1 % kStages, fill = 0;
  for (int c = c0; c < c1; ++c) {
    if (rank > 0 && c + kStages - 1 < c1) stage_expand<R>(s.ring[fill][warp], wb, c + kStages - 1, rs, lane);
    cp_async_commit();
    const bool in = 32 * c + 8 * q < p.N;
    Raw8<E> b[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (p.base && p.out_vec && in && (live >> (2 * m + h) & 1u))
          b[m][h].load(base[m][h] + 32 * c);
        else
          b[m][h].zero();
      }
    cp_async_wait<kStages - 1>();
    __syncwarp();  // (the products are the whole warp's, and lanes without a row skipped the stores before them)
    const uint4* w = reinterpret_cast<const uint4*>(s.ring[slot][warp]) + lane;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float acc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
      if (rank > 0) {
#pragma unroll
        for (int k = 0; k < RS; ++k)
          if (k < rs) {
            const uint4 w0 = w[2 * k * 32], w1 = w[(2 * k + 1) * 32];
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
              const uint2 a0 = kHold ? u[kHold ? m : 0][kHold ? k : 0][t][0]
                                     : *reinterpret_cast<const uint2*>(&s.u[t][16 * m + g][16 * k + 4 * q]);
              const uint2 a1 = kHold ? u[kHold ? m : 0][kHold ? k : 0][t][1]
                                     : *reinterpret_cast<const uint2*>(&s.u[t][16 * m + g + 8][16 * k + 4 * q]);
              mma<kFp16>(acc[0], a0.x, a1.x, a0.y, a1.y, w0.x, w0.y);
              mma<kFp16>(acc[1], a0.x, a1.x, a0.y, a1.y, w0.z, w0.w);
              mma<kFp16>(acc[2], a0.x, a1.x, a0.y, a1.y, w1.x, w1.y);
              mma<kFp16>(acc[3], a0.x, a1.x, a0.y, a1.y, w1.z, w1.w);
            }
          }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!(live >> (2 * m + h) & 1u)) continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = acc[j][2 * h], v[2 * j + 1] = acc[j][2 * h + 1];
        if (p.out_vec) {
          float f[8];
          b[m][h].to_f32(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = kFp16 ? fmaf(v[i], mul[m][h], f[i]) : v[i] + f[i];
          if (in) {
            if (rank > 0)  // (else the base's bits as they are: a sum would change -0 and NaN)
              store8(out[m][h] + 32 * c, v);
            else
              b[m][h].store(out[m][h] + 32 * c);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (32 * c + 8 * q + i < p.N) {
              const E e = p.base ? base[m][h][32 * c + i] : E{};
              const float f = e.f32();
              out[m][h][32 * c + i] = rank == 0 ? e : E::of(kFp16 ? fmaf(v[i], mul[m][h], f) : v[i] + f);
            }
        }
      }
    }
    slot = slot + 1 == kStages ? 0 : slot + 1;
    fill = fill + 1 == kStages ? 0 : fill + 1;
  }
}

template <int M, int R, bool kFp16>
__global__ void __launch_bounds__(kThreads, 2) adapter_kernel(const AdapterArgs p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<M, R, kFp16>& s = *reinterpret_cast<Smem<M, R, kFp16>*>(smem_raw);
  constexpr int MT = M / 16, NT = R / 8, kStages = Smem<M, R, kFp16>::kStages, kSlots = Smem<M, R, kFp16>::kSlots;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  pdl_trigger();
  pdl_wait();
  int slot, rank;
  if (!find_tile(p, s, slot, rank)) return;
  if (rank == 0 && p.base == p.out) return;
  const int cta = cluster_rank(), C = p.cut.ctas;
  // this warp's chunks of 32 features
  const int nc = (p.N + 31) / 32, per_n = (nc + C * kWarps - 1) / (C * kWarps);
  const int c0 = min((cta * kWarps + warp) * per_n, nc), c1 = min(c0 + per_n, nc);
  const uint4* wb = reinterpret_cast<const uint4*>(p.b + (rank > 0 ? slot * p.b_slot : 0)) + lane;

  if (rank > 0) {
    // ---- shrink: this warp's chunks of 32 columns ---------------------------------------------------
    const int nt = (rank + 7) / 8;
    const int nk = (p.K + 31) / 32, per = (nk + C * kWarps - 1) / (C * kWarps);
    const int k0 = min((cta * kWarps + warp) * per, nk), k1 = min(k0 + per, nk);
    const uint4* wa = reinterpret_cast<const uint4*>(p.a + slot * p.a_slot) + lane;
    const uint16_t* x_row[MT][2];  // (rows past the tile's last read its first: their results go nowhere)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = s.rows[16 * m + g + 8 * h];
        x_row[m][h] = p.x + (r >= 0 ? r : s.rows[0]) * p.ldx + 8 * q;
      }
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[m][j][0] = acc[m][j][1] = acc[m][j][2] = acc[m][j][3] = 0.0f;
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
      if (k0 + i < k1) stage_shrink<M, R>(p, s.ring[i][warp], x_row, wa, k0 + i, nt, lane);
      cp_async_commit();
    }
    int from = 0, fill = kStages - 1;
    for (int k = k0; k < k1; ++k) {
      if (k + kStages - 1 < k1) stage_shrink<M, R>(p, s.ring[fill][warp], x_row, wa, k + kStages - 1, nt, lane);
      cp_async_commit();
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint4* st = reinterpret_cast<const uint4*>(s.ring[from][warp]) + lane;
      uint4 x[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m) x[m][0] = st[2 * m * 32], x[m][1] = st[(2 * m + 1) * 32];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (j < nt) {
          const uint4 w = st[(M / 8 + j) * 32];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            mma<kFp16>(acc[m][j], x[m][0].x, x[m][1].x, x[m][0].y, x[m][1].y, w.x, w.y);
            mma<kFp16>(acc[m][j], x[m][0].z, x[m][1].z, x[m][0].w, x[m][1].w, w.z, w.w);
          }
        }
      from = from + 1 == kStages ? 0 : from + 1;
      fill = fill + 1 == kStages ? 0 : fill + 1;
    }
    __syncthreads();  // no warp reads its ring any more
    // B's first chunks are on their way while u is put together (into the stages that hold no sums)
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
      if (c0 + i < c1) stage_expand<R>(s.ring[i + 1][warp], wb, c0 + i, (rank + 15) / 16, lane);
      cp_async_commit();
    }
    // ---- u: the warps' sums in pairs, then the pairs, then the CTAs, in order ---------------------------
    if (warp >= kSlots) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float(*o)[R] = s.warp_part[warp - kSlots];
          *reinterpret_cast<float2*>(&o[16 * m + g][8 * j + 2 * q]) = make_float2(acc[m][j][0], acc[m][j][1]);
          *reinterpret_cast<float2*>(&o[16 * m + g + 8][8 * j + 2 * q]) = make_float2(acc[m][j][2], acc[m][j][3]);
        }
    }
    __syncthreads();
    if (warp < kSlots) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float(*o)[R] = s.warp_part[warp];
          float2* lo = reinterpret_cast<float2*>(&o[16 * m + g][8 * j + 2 * q]);
          float2* up = reinterpret_cast<float2*>(&o[16 * m + g + 8][8 * j + 2 * q]);
          *lo = make_float2(acc[m][j][0] + lo->x, acc[m][j][1] + lo->y);
          *up = make_float2(acc[m][j][2] + up->x, acc[m][j][3] + up->y);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x * 4; i < M * R; i += kThreads * 4) {
      float4 v = *reinterpret_cast<const float4*>(&s.warp_part[0][0][0] + i);
#pragma unroll
      for (int w = 1; w < kSlots; ++w) {
        const float4 o = *reinterpret_cast<const float4*>(&s.warp_part[w][0][0] + i);
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
      }
      *reinterpret_cast<float4*>(&s.part[0][0] + i) = v;
    }
    cluster_barrier();
    const float scale = p.slots.scale[slot];
    for (int i = threadIdx.x * 8; i < M * R; i += kThreads * 8) {  // eight ranks a thread
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      const uint32_t at = smem_u32(&s.part[0][0] + i);
      for (int c = 0; c < C; c += 4) {  // four CTAs' sums in flight
        float4 o[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[e][0] = o[e][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c + e < C) {
            const uint32_t from = cluster_addr_u32(at, c + e);
            o[e][0] = ld_cluster_f32x4(from), o[e][1] = ld_cluster_f32x4(from + 16);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[0] += o[e][0].x, v[1] += o[e][0].y, v[2] += o[e][0].z, v[3] += o[e][0].w;
          v[4] += o[e][1].x, v[5] += o[e][1].y, v[6] += o[e][1].z, v[7] += o[e][1].w;
        }
      }
      const int r = i / R, c = i % R;
      uint4 term[kAdapterTerms<kFp16>];
      const float mul = adapter_split<R, kFp16>(v, c, rank, scale, term);
      if (kFp16 && c == 0) s.row_scale[r] = mul;
#pragma unroll
      for (int t = 0; t < kAdapterTerms<kFp16>; ++t) *reinterpret_cast<uint4*>(&s.u[t][r][c]) = term[t];
    }
    cluster_barrier();  // u is written, and no CTA's partial sums are read any more
  }
  if (p.out_type == MOE_BF16)
    expand<Bf16, M, R, kFp16>(p, s, wb, c0, c1, rank, lane, warp);
  else if (p.out_type == MOE_FP16)
    expand<Fp16, M, R, kFp16>(p, s, wb, c0, c1, rank, lane, warp);
  else
    expand<Fp32, M, R, kFp16>(p, s, wb, c0, c1, rank, lane, warp);
}

// ---- packing -------------------------------------------------------------------------------------------
// A: for a chunk of 32 columns and 8 ranks, lane (g, q) holds rank 8 j + g, columns 8 q .. 8 q + 7.
// B: for a chunk of 32 features and 16 ranks, lane (g, q) holds, for each of the four products t, feature
// 8 (g / 2) + 2 t + g % 2, ranks 4 q .. 4 q + 3.
__global__ void adapter_pack_kernel(const uint16_t* a, const uint16_t* b, uint16_t* pa, uint16_t* pb, int r, int K, int N,
                                    int R, int64_t na, int64_t nb) {
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < na + nb;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    if (i < na) {
      const int e = i % 8, lane = i / 8 % 32, j = i / 256 % (R / 8);
      const int64_t chunk = i / 256 / (R / 8);
      const int rank = 8 * j + lane / 4;
      const int64_t col = 32 * chunk + 8 * (lane % 4) + e;
      pa[i] = rank < r && col < K ? a[rank * static_cast<int64_t>(K) + col] : 0;
    } else {
      const int64_t o = i - na;
      const int e = o % 4, t2 = o / 4 % 2, lane = o / 8 % 32, half = o / 256 % 2, k = o / 512 % (R / 16);
      const int64_t chunk = o / 512 / (R / 16);
      const int g = lane / 4, q = lane % 4, t = 2 * half + t2, rank = 16 * k + 4 * q + e;
      const int64_t f = 32 * chunk + 8 * (g / 2) + 2 * t + g % 2;
      pb[o] = rank < r && f < N ? b[f * r + rank] : 0;
    }
  }
}

// ---- grouping of larger steps -----------------------------------------------------------------------------
// The rows in slot order and their tiles, from ids, by one cluster: each CTA counts the ids of its share of the rows
// (no adapter counts as slot n), the counts meet in distributed shared memory, every CTA scans all slots' rows and
// tiles, and places its rows.  The order of a slot's rows is not fixed; a row's result does not depend on its place.
constexpr int kGroupThreads = 1024;
constexpr int kGroupCtas = 8;
__global__ void __launch_bounds__(kGroupThreads) adapter_group_kernel(const int32_t* ids, int T, int n, int ctas,
                                                                      int fit, const AdapterSlots slots,
                                                                      int32_t* order, AdapterTile* tiles,
                                                                      int32_t* n_tiles, uint32_t* err) {
  __shared__ int s_count[kAdaptersMax + 1];                                             // of this CTA's rows
  __shared__ int s_all[kAdaptersMax + 1], s_first[kAdaptersMax + 1], s_tile[kAdaptersMax + 1];  // of the slot
  __shared__ int s_next[kAdaptersMax + 1];                                              // this CTA's next place
  __shared__ int s_warp[2][32], s_tiles[kAdapterTileRows / 16];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = cluster_rank();
  for (int i = tid; i <= n; i += kGroupThreads) s_count[i] = 0;
  if (tid < kAdapterTileRows / 16) s_tiles[tid] = 0;
  __syncthreads();
  bool bad_id = false;
  for (int i0 = cta * kGroupThreads; i0 < T; i0 += kGroupCtas * kGroupThreads) {
    const int i = i0 + tid;
    int key = -1;
    if (i < T) {
      key = ids[i];
      if (key < 0 || key >= n) bad_id |= key != -1, key = n;
    }
    count_key(s_count, key, lane);
  }
  if (bad_id) set_error(err, MOE_DEVERR_EXPERT_RANGE);
  cluster_barrier();
  // slot tid: its rows in all CTAs, and in the CTAs before this one; inclusive scans of rows and tiles
  int c = 0, before = 0;
  if (tid <= n) {
    int v[kGroupCtas];
#pragma unroll
    for (int k = 0; k < kGroupCtas; ++k) v[k] = ld_cluster_s32(cluster_addr(&s_count[tid], k));
#pragma unroll
    for (int k = 0; k < kGroupCtas; ++k) {
      c += v[k];
      if (k < cta) before += v[k];
    }
  }
  // Rows of a tile: as few (64 to 128, in steps of 16) as leave the number of waves that 128 would need
  constexpr int kSizes = kAdapterTileRows / 16;
  const int of_slot = tid < n ? c : 0;
#pragma unroll
  for (int m = 3; m < kSizes; ++m) {
    int v = (of_slot + 16 * m + 15) / (16 * m + 16);
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && v) atomicAdd(&s_tiles[m], v);
  }
  __syncthreads();
  int M = kAdapterTileRows;
  const int64_t waves = (static_cast<int64_t>(s_tiles[kSizes - 1]) * ctas + fit - 1) / fit;
  for (int m = kSizes - 2; m >= 3; --m)
    if (static_cast<int64_t>(s_tiles[m]) * ctas <= waves * fit) M = 16 * m + 16;
  int r = c, t = (of_slot + M - 1) / M;
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, r, o), b = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) r += a, t += b;
  }
  if (lane == 31) s_warp[0][warp] = r, s_warp[1][warp] = t;
  __syncthreads();
  for (int w = 0; w < warp; ++w) r += s_warp[0][w], t += s_warp[1][w];
  if (tid <= n) s_all[tid] = c, s_first[tid] = r - c, s_tile[tid] = t - (of_slot + M - 1) / M, s_next[tid] = r - c + before;
  if (n == kGroupThreads && tid == kGroupThreads - 1) {  // the rows without an adapter, behind the last thread's slot
    int mine = 0;
    for (int k = 0; k < cta; ++k) mine += ld_cluster_s32(cluster_addr(&s_count[n], k));
    s_first[n] = r, s_next[n] = r + mine;
  }
  __syncthreads();
  if (cta == 0 && tid == kGroupThreads - 1) n_tiles[0] = t, n_tiles[1] = s_first[n], n_tiles[2] = M;
  cluster_barrier();  // (also: no CTA reads another's counts any more)
  for (int i0 = cta * kGroupThreads; i0 < T; i0 += kGroupCtas * kGroupThreads) {
    const int i = i0 + tid;
    int key = -1;
    if (i < T) {
      key = ids[i];
      if (key < 0 || key >= n) key = n;
    }
    const int at = count_key(s_next, key, lane);
    if (key < 0) continue;
    order[at] = i;
    if (key == n) continue;
    const int in = at - s_first[key];
    const int all = s_all[key], per = adapter_tile_rows(all, M);  // the row that comes first in a tile writes the tile
    if (in % per == 0) {
      const AdapterTile t{key, at, static_cast<uint16_t>(min(per, all - in)), static_cast<uint16_t>(slots.rank[key]),
                          slots.scale[key]};
      tiles[s_tile[key] + in / per] = t;
    }
  }
}

// One cluster for each tile that there may be, of as many CTAs (1 to 8) as run at the same time.
template <int R, bool kFp16>
cudaError_t launch(AdapterArgs p, int num_sms, cudaStream_t st) {
  auto kern = adapter_kernel<kTileRows, R, kFp16>;
  const int smem = sizeof(Smem<kTileRows, R, kFp16>);
  cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int most = (p.n + 1 < p.T ? p.n + 1 : p.T) + p.T / kTileRows, tiles = most < p.T ? most : p.T;
  const int fit = (R <= 64 ? 2 : 1) * num_sms / tiles;
  p.cut.ctas = fit < 1 ? 1 : fit > 8 ? 8 : fit;
  return launch_pdl_clusters(kern, dim3(tiles * p.cut.ctas), dim3(kThreads), p.cut.ctas, smem, st, p);
}

template <int R>
cudaError_t launch_rank(const AdapterArgs& p, bool fp16, int num_sms, cudaStream_t st) {
  return fp16 ? launch<R, true>(p, num_sms, st) : launch<R, false>(p, num_sms, st);
}

}  // namespace

cudaError_t launch_adapter_pack(const uint16_t* a, const uint16_t* b, uint16_t* pa, uint16_t* pb, int r, int K, int N,
                                int rpad, cudaStream_t st) {
  const int64_t na = adapter_a_elems(K, rpad), nb = adapter_b_elems(N, rpad);
  const int64_t blocks = (na + nb + 255) / 256;
  adapter_pack_kernel<<<static_cast<int>(blocks < 4096 ? blocks : 4096), 256, 0, st>>>(a, b, pa, pb, r, K, N, rpad, na, nb);
  return cudaGetLastError();
}

cudaError_t launch_adapter_group(const int32_t* ids, int T, int n, const AdapterCut& cut, const AdapterSlots& slots, int32_t* order,
                                 AdapterTile* tiles, int32_t* n_tiles, uint32_t* err, cudaStream_t st) {
  return launch_pdl_clusters(adapter_group_kernel, dim3(kGroupCtas), dim3(kGroupThreads), kGroupCtas, 0, st, ids, T, n,
                             cut.ctas, cut.slots, slots, order, tiles, n_tiles, err);
}

cudaError_t launch_adapters(const AdapterArgs& p, int rpad, bool fp16, int num_sms, cudaStream_t st) {
  switch (rpad) {
    case 16: return launch_rank<16>(p, fp16, num_sms, st);
    case 32: return launch_rank<32>(p, fp16, num_sms, st);
    case 64: return launch_rank<64>(p, fp16, num_sms, st);
    default: return launch_rank<128>(p, fp16, num_sms, st);
  }
}

}  // namespace moe
