// 8-bit block-scaled GEMMs on the 5th-generation tensor cores (tcgen05 kind::f8f6f4), sm_103a.
//
//     out[r][n] = sum_b  sa[r][b] * sw[n / 128][b] * ( sum_{k in block b} a[r][k] * w[n][k] )
//
// a: e4m3 rows with one fp32 scale per 128 elements; w: e4m3 with one fp32 scale per 128 x 128.  The
// scales are arbitrary fp32 numbers, so the sum over blocks cannot stay in the tensor core's
// accumulator: each K block of 128 (four MMAs of K = 32) makes a fresh accumulator in TMEM, and the
// epilogue warps add it, times its scale, to fp32 sums that they hold in registers for the whole K
// loop.  The rows of `a` are the MMA's M (TMEM lanes), the weight rows its N: a thread owns one row
// of `a`, so a block has one scale for all of the thread's columns that share a weight block.
//
// Uses of one kernel:
//   gate/up  a = rows of x gathered by the permutation; a tile's 256 weight rows are two times (64
//            gate rows, the same 64 features' up rows); the epilogue forms silu(g) * u in fp32,
//            quantises the 128 features (one activation block of h) and writes codes and scale.
//   down     a = those rows of h; y in fp16 in grouped order for the combine.
//   linear   a = the T rows of one matrix; bf16 or fp32 out.  Sets of 32 whole bf16 rows leave by TMA stores that
//            nobody waits for.
//   split    linear with few units: a cluster of S CTAs shares a unit, each a range of its K blocks;
//            the fp32 sums meet in shared memory and every CTA adds up (in split order) and writes a
//            1/S of the columns.
// Routed units are ordered tile-major within an expert's parts, linear units tile-major over the
// row parts: CTAs that share a weight tile run side by side and its second read is served by L2.
//
// What bounds them, measured on a GB300 (6.78 TB/s copy, 1.94 PFLOP/s bf16): up to about 100 rows an expert
// the weight stream (256 experts, d 2048, f 512, 2051 tokens x 8: gate/up 91 us at 6.0 TB/s, down 55 us at
// 5.2 TB/s); 8192 x 4096 x 4096, 111 us, 2.5 PFLOP/s, three things at once: the MMAs (512 cycles a K block), the
// epilogue's additions (64 packed FMAs a thread at two cycles, and as many TMEM loads) and the operands'
// way from L2 (48 KB a block, 768 cycles at 64 bytes a cycle).  Without the results' stores any two of them
// take 89 to 96 us and all three 101; full tiles of gate/up (8 experts of 2051 rows, d 4096, f 1024: 166 us,
// 1.65 PFLOP/s) the additions and the row gather: 139 us without the gather's copies, 95 without the additions
// as well; few rows, latency.
//
// Roles (persistent CTAs, one per SM, every role walks the same unit sequence):
//   warp 0      producer: weights by bulk copy (tile-contiguous, pre-swizzled); rows by TMA
//   warp 1      TMEM owner and MMA issuer
//   warp 2      unit list: decodes the CTA's units ahead of the other roles into a ring of shared-memory
//               records (gate/up: with the source row of each grouped row), so that no role waits for
//               a chain of global loads where one unit follows the other
//   warp 3      scales: asynchronous copies of the rows' and the weight blocks' scales into shared memory,
//               in groups of four K blocks, up to four groups ahead of the epilogue (which has no
//               registers to hold them in; with a load one block ahead its latency set the pace)
//   warps 4-11  epilogue: warps 4-7 the tile's first half, 8-11 the second; TMEM lanes 32 (warp % 4)
//   warps 12-15 gate/up: cp.async gather of the rows, one warp per stage slot
// Registers move from the first (and the gather) warps to the epilogue warps, which hold 128 sums a
// thread.  TMEM: two buffers of 256 columns, so one block's MMAs overlap the previous block's sums.
// Rows of a tile beyond the segment's are never copied: whatever the slot held lands in lanes that
// nobody reads.
#include "fp8.cuh"
#include "kernels.h"

#include <map>
#include <mutex>

namespace moe {
namespace f8 {

constexpr int kGateUp = 0, kDown = 1, kLinear = 2, kSplit = 3;
constexpr int BM = 128;                           // activation rows per tile (MMA M)
constexpr int kBBytes = 2 * kF8TileBytes;         // 256 weight rows x 128 K elements
constexpr int kABytes = BM * kF8Block;
constexpr int kStageBytes = kABytes + kBBytes;    // 48 KB
constexpr int kAccCols = 256;
constexpr int kTmemCols = 2 * kAccCols;
constexpr int kEpiWarps = 8, kFirstEpi = 4, kFirstGather = 12;
constexpr int kRing = 4;                          // decoded units
constexpr uint32_t kSpinLimit = 1u << 20;         // tries of an epilogue wait: 1.4 s at 1.3 us a try
constexpr int kScGroups = 4;                      // groups of four K blocks of scales
constexpr int kScGroupBytes = BM * 16 + 32;       // a row's four scales; the tile's four pairs
constexpr int kScaleBytes = kScGroups * kScGroupBytes;
constexpr int kTokBytes = kRing * BM * 4;         // gate/up, per unit: source row of each row
constexpr int kXchBytes = 2 * 2 * BM * 4;         // gate/up, row maxima of h: [unit parity][half][row]
constexpr int kOutPitch = 64 + 16;                // a staged row of results: 64 bytes, odd in 16-byte units
constexpr int kOutBytes = 32 * kOutPitch;         // per epilogue warp
constexpr int kTmaOutBytes = 2 * 32 * 128;        // linear: two boxes of 32 rows x 128 bytes
constexpr int kSumPitch = 256 * 4 + 16;           // split: a row of fp32 sums (in the stages' space)
static_assert(BM * kSumPitch <= 3 * kStageBytes, "sums in the stages");

template <int kMode>
struct Cfg {
  // linear trades a stage for staging space of whole bf16 results, which TMA stores read while the next
  // unit is under way (8192 x 4096 x 4096 with the quantisation: 126-130 us; four stages and row pieces 133;
  // four stages and boxes of 32 columns through 2 KB, waited for in between, 134; without any stores 114)
  static constexpr int kStages = kMode == kLinear ? 3 : 4;
  static constexpr int kExtra = kMode == kGateUp ? kTokBytes + kXchBytes : kMode == kLinear ? kEpiWarps * kTmaOutBytes
                                                                                        : kEpiWarps * kOutBytes;
  static constexpr int kSmemBytes = kStages * kStageBytes + 1024 /*barriers*/ + 1024 /*align slack*/ + kScaleBytes + kExtra;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static constexpr int kThreads = kMode == kGateUp ? 512 : 384;
  // register split: the sums over the warpgroups equal the launch's (128 x 4 or 168 x 3)
  static constexpr int kRegsEpi = kMode == kGateUp ? 200 : 216;
  static constexpr int kRegsRest = kMode == kGateUp ? 56 : 72;
  // warps that read each unit record: producer, MMA, scales, epilogue, gather
  static constexpr int kReaders = 3 + kEpiWarps + (kMode == kGateUp ? kStages : 0);
};

struct Unit {
  int expert, row_start, rows, tile;  // rows == 0: the CTA's units are done
};

MOE_DEVICE Seg load_seg(const Seg* p) {  // through L2: read before the grid-dependency wait (down)
  const int4 lo = __ldcg(reinterpret_cast<const int4*>(p));
  const int4 hi = __ldcg(reinterpret_cast<const int4*>(p) + 1);
  return Seg{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

// Part p of `parts` near-equal parts of `total` rows.
MOE_DEVICE void part_of(int total, int parts, int p, int& first, int& rows) {
  const int q = total / parts, rem = total % parts;
  first = p * q + min(p, rem);
  rows = q + (p < rem ? 1 : 0);
}

template <int kMode>
MOE_DEVICE Unit decode_unit(int u, const F8Args& a, int tiles) {
  Unit un;
  if (kMode >= kLinear) {
    const int parts = (a.T + BM - 1) / BM;
    un.expert = 0;
    un.tile = u / parts;
    part_of(a.T, parts, u % parts, un.row_start, un.rows);
  } else {
    const Seg s = load_seg(a.segs + u / tiles);
    const int o = u - s.first * tiles;
    un.expert = s.expert;
    un.tile = o / s.nparts;
    part_of(s.total, s.nparts, o % s.nparts, un.row_start, un.rows);
    un.row_start += s.start;
  }
  return un;
}

// The unit of a CTA's step when half of the CTAs go through the list from its front and half from its
// back, in turns (total: none is left).  Experts with many rows keep the epilogue busy (their parts share
// weights through L2), experts with few rows the memory; where busy experts lie together, front to back
// would run one kind after the other.  Zipf layer, T = 2051, front to back / from both ends: popularity
// along the expert index 494 / 460 us, against it 502 / 459; popular experts anywhere (four permutations)
// 468, 455, 461, 453 / 475, 466, 468, 476.  So this order costs up to 5% where experts are mixed already and
// saves 7 to 9% where they are not; uniform load is the same.  Neighbouring units still run side by side.
// An odd grid goes front to back.
MOE_DEVICE int mixed_unit(int step, int total) {
  if (gridDim.x & 1) return min(static_cast<int>(blockIdx.x + step * gridDim.x), total);
  const int o = step * static_cast<int>(gridDim.x / 2) + static_cast<int>(blockIdx.x / 2);
  if (((step ^ static_cast<int>(blockIdx.x)) & 1) == 0) return o < (total + 1) / 2 ? o : total;
  return o < total / 2 ? total - 1 - o : total;
}

// The ring of decoded units: record j is read by every role's warps.
struct Ring {
  uint64_t *full, *empty;
  const int4* rec;
  volatile int* abort_flag;
  uint32_t* err;
  // Record j once it is there; a record without rows ends the loop (as does an expired wait).
  MOE_DEVICE Unit get(uint32_t j) const {
    if (!mbar_wait_warp(&full[j % kRing], (j / kRing) & 1u, abort_flag, err)) return Unit{0, 0, 0, 0};
    const int4 v = rec[j % kRing];  // (the wait is a compiler barrier too)
    return Unit{v.x, v.y, v.z, v.w};
  }
  // The calling warp no longer reads record j (nor the row table beside it).
  MOE_DEVICE void done(uint32_t j) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[j % kRing]);
  }
};

// Adds 128 columns of one K block, times the scales (s01 the first 64 columns', s23 the rest's), to
// the thread's sums: 16-column loads, one in flight while the previous one is added.
// The buffer is handed back once the last load is in registers.
MOE_DEVICE void add_block(uint64_t (&acc)[64], uint32_t taddr, uint64_t s01, uint64_t s23, uint32_t empty) {
  uint32_t r[2][16];
  tmem_ld_32x32b_x16(taddr, r[0]);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    tmem_wait_ld(s01, s23);
    if (c < 7) {
      tmem_ld_32x32b_x16(taddr + 16 * (c + 1), r[(c + 1) & 1]);
    } else {
      tc_fence_before();
      __syncwarp();
      mbar_arrive_lane0_u32(empty);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      fma_f32x2(acc[8 * c + i], pack_f32x2(__uint_as_float(r[c & 1][2 * i]), __uint_as_float(r[c & 1][2 * i + 1])),
                c < 4 ? s01 : s23);
  }
}

MOE_DEVICE void st_global_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Cluster barrier of every thread (arrive.release, wait.acquire), and 16 bytes of CTA `rank`'s shared memory
// at this CTA's address `addr`.
MOE_DEVICE void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
MOE_DEVICE float4 ld_cluster_v4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}
// TMA store of a box (64 x 32 elements, 128-byte swizzled in shared memory) at column c0, row c1; the bulk
// groups of the issuing thread.
MOE_DEVICE void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(src)
               : "memory");
}
MOE_DEVICE void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
MOE_DEVICE void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
MOE_DEVICE void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
MOE_DEVICE float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
MOE_DEVICE float2 ld_shared_v2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
MOE_DEVICE uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
MOE_DEVICE uint16_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
MOE_DEVICE uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
MOE_DEVICE void st_shared_v4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Writes the warp's first `rows` staged rows, `cols` elements each, to out at (row0, col).  4 lanes take a
// row's 64 bytes where rows and columns allow 16-byte stores, else 32 lanes one element each (8192 rows,
// K = 1000, bf16 / fp32 out, quantisation included: N = 1344 23 / 31 us, N = 1337 36 / 58).
template <typename E>
MOE_DEVICE void send_rows(const F8Args& a, uint32_t stage, int64_t row0, int rows, int64_t col, int cols, uint64_t pol) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  if (a.out_vec) {
    const int c = (lane & 3) * (16 / static_cast<int>(sizeof(E)));
    if (c < cols) {
      E* o = static_cast<E*>(a.out) + (row0 + (lane >> 2)) * a.ldo + col + c;
      const uint32_t src = stage + (lane >> 2) * kOutPitch + (lane & 3) * 16;
#pragma unroll
      for (int i = 0; i < 32; i += 8)
        if (i + (lane >> 2) < rows) st_global_v4_hint(o + static_cast<int64_t>(i) * a.ldo, ld_shared_v4(src + i * kOutPitch), pol);
    }
  } else {
    for (int i = 0; i < rows; ++i) {
      E* o = static_cast<E*>(a.out) + (row0 + i) * a.ldo + col;
      for (int c = lane; c < cols; c += 32) {
        if (sizeof(E) == 2)
          *reinterpret_cast<uint16_t*>(o + c) = ld_shared_u16(stage + i * kOutPitch + 2 * c);
        else
          *reinterpret_cast<uint32_t*>(o + c) = ld_shared_u32(stage + i * kOutPitch + 4 * c);
      }
    }
  }
  __syncwarp();
}

// The warp's rows row0 .. row0 + rows - 1 (a lane each; beyond 32 or below 1 clipped), 128 columns from
// col0 (of N), through its staging space.
template <int kMode>
MOE_DEVICE void store_rows(const uint64_t (&acc)[64], const F8Args& a, const CUtensorMap* omap, uint32_t stage,
                           int64_t row0, int rows, int col0, uint64_t pol) {
  const int n = min(128, a.N - col0);  // valid columns here
  const uint32_t mine = stage + (threadIdx.x & 31) * kOutPitch;
  rows = min(rows, 32);
  if (kMode == kLinear) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) bulk_wait_read();  // an earlier TMA store still reads the staging space
    __syncwarp();
    // 32 whole rows leave as two TMA stores of 64 columns, which nobody waits for (128-byte swizzled
    // staging rows); a partial set of rows, whose neighbours belong to others, as row pieces
    if (a.out_vec && rows == 32 && a.out_type == MOE_BF16) {
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo, hi;
          unpack_f32x2(acc[4 * c + i], lo, hi);
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
        }
        st_shared_v4(stage + lane * 128 + (c >> 3) * 4096 + (((c & 7) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(omap, stage, col0, static_cast<int>(row0));
        if (n > 64) tma_store_2d(omap, stage + 4096, col0 + 64, static_cast<int>(row0));
        bulk_commit();
      }
      return;
    }
  }
  if (kMode == kDown || a.out_type == MOE_BF16) {
    float m = 0.f;
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // 32 columns at a time
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo, hi;
          unpack_f32x2(acc[16 * h + 4 * c + i], lo, hi);
          if (kMode == kDown) {
            // y in fp16, what the experts' entry returns and the combine reads, for every weight type: half the
            // bytes of fp32.  2e-4 of its size (rms), 9e-4 after the layer's bf16 rounding, where other orders
            // of the fp32 sums alone give 4e-4 by h's open roundings; from fp64 1.67e-3 with it and without.
            m = fmaxf(m, fmaxf(fabsf(lo), fabsf(hi)));  // (columns beyond N have zero weights)
            w[i] = f32x2_to_f16x2_sat(lo, hi);
          } else {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
          }
        }
        st_shared_v4(mine + 16 * c, w[0], w[1], w[2], w[3]);
      }
      send_rows<uint16_t>(a, stage, row0, rows, col0 + 32 * h, min(32, n - 32 * h), pol);
    }
    if (kMode == kDown && m > kF16Max && static_cast<int>(threadIdx.x & 31) < rows) set_error(a.err, MOE_DEVERR_RANGE);
  } else {
#pragma unroll
    for (int h = 0; h < 8; ++h) {  // 16 columns at a time
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float v[4];
        unpack_f32x2(acc[8 * h + 2 * c], v[0], v[1]);
        unpack_f32x2(acc[8 * h + 2 * c + 1], v[2], v[3]);
        st_shared_v4(mine + 16 * c, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      }
      send_rows<uint32_t>(a, stage, row0, rows, col0 + 16 * h, min(16, n - 16 * h), pol);
    }
  }
}

template <int kMode>
__global__ void __launch_bounds__(Cfg<kMode>::kThreads, 1)
    f8_gemm_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap amap128,
                   const __grid_constant__ CUtensorMap omap, const F8Args a) {
  constexpr int kStages = Cfg<kMode>::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* extra = smem + kStages * kStageBytes;
  int32_t* tok_tab = reinterpret_cast<int32_t*>(extra);                         // gate/up
  volatile float* xch = reinterpret_cast<volatile float*>(extra + kTokBytes);   // gate/up
  uint8_t* out_tab = extra;                                                     // linear, down
  uint8_t* bars = extra + Cfg<kMode>::kExtra;
  uint64_t* full = reinterpret_cast<uint64_t*>(bars);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* xch_bar = acc_empty + 2;   // per lane quarter: both halves published their row maxima
  uint64_t* ring_full = xch_bar + 4;
  uint64_t* ring_empty = ring_full + kRing;
  uint64_t* sc_full = ring_empty + kRing;
  uint64_t* sc_empty = sc_full + kScGroups;
  uint64_t* drain = sc_empty + kScGroups;
  int4* ring_rec = reinterpret_cast<int4*>(bars + 512);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* sc_tab = bars + 1024;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], kMode == kGateUp ? 2 : 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&xch_bar[q], 2);
    for (int i = 0; i < kScGroups; ++i) {
      mbar_init(&sc_full[i], 32);  // each lane's copies
      mbar_init(&sc_empty[i], kEpiWarps);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&ring_full[i], 1);
      mbar_init(&ring_empty[i], Cfg<kMode>::kReaders);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0 && kMode != kGateUp) tma_prefetch_map(&amap);
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // gate/up lets its dependents start only once the routing is complete, so the down kernel may
  // read the segment list and stream its first weight stages before its grid-dependency wait;
  // linear's weights depend on nothing.  Everything that reads activations waits.
  if (kMode == kGateUp) {
    pdl_wait();
    pdl_trigger();
  } else {
    pdl_trigger();
    if (warp != 0 && warp != 2) pdl_wait();  // the unit list and the weights are there already
  }

  const int tiles = (a.halves + 1) / 2;
  const int nk = a.nk;
  // split: this CTA's share of the K blocks
  const int split = kMode == kSplit ? static_cast<int>(blockIdx.x) % a.splits : 0;
  const int kb0 = kMode == kSplit ? split * nk / a.splits : 0;
  const int kb1 = kMode == kSplit ? (split + 1) * nk / a.splits : nk;
  const Ring ring{ring_full, ring_empty, ring_rec, abort_flag, a.err};

  if (warp < kFirstEpi) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg<kMode>::kRegsRest));
    if (warp == 0) {
      // ---------------- producer ----------------
      const uint64_t pol_w = l2_policy_evict_first();
      const uint64_t pol_act = l2_policy_evict_last();
      uint32_t pre = 0;  // stages whose weights were requested before the dependency wait
      if (kMode != kGateUp) {
        // (at most kStages units, whose records stay in the ring until the main loop has read them)
        for (uint32_t j = 0; pre < static_cast<uint32_t>(kStages); ++j) {
          const Unit un = ring.get(j);
          if (un.rows == 0) break;
          const int ntile = min(2, a.halves - 2 * un.tile);
          const uint8_t* wb = a.w + un.expert * a.w_stride;
          for (int kb = kb0; kb < kb1 && pre < static_cast<uint32_t>(kStages); ++kb, ++pre) {
            if (elect_one()) {  // a fresh slot: no wait; the arrival comes with the rows below
              mbar_expect_tx(&full[pre], ntile * kF8TileBytes);
              bulk_load(smem + pre * kStageBytes, wb + f8_half_offset(2 * un.tile, kb, a.halves, nk), ntile * kF8TileBytes,
                        &full[pre], pol_w);
            }
            __syncwarp();
          }
        }
        pdl_wait();
      }
      // One elected lane runs a unit's K loop (as the MMA issuer does): with a vote and four row loads
      // a block the producer was as slow as the epilogue.
      const uint32_t full0 = smem_u32(full), base0 = smem_u32(smem);
      uint32_t g = 0;
      bool ok = true;
      for (uint32_t j = 0; ok; ++j) {
        const Unit un = ring.get(j);
        if (un.rows == 0) break;
        ring.done(j);
        const uint32_t wbytes = min(2, a.halves - 2 * un.tile) * kF8TileBytes;
        const uint8_t* wp = a.w + un.expert * a.w_stride + f8_half_offset(2 * un.tile, kb0, a.halves, nk);
        // rows by boxes of a.box_rows (linear: a part's rows in one box), or of 128 where that many are wanted
        const bool big = kMode == kDown && un.rows > 64;
        const int box = big ? BM : a.box_rows;
        const int nbox = kMode == kGateUp ? 0 : (un.rows + box - 1) / box;
        const uint32_t abytes = nbox * box * kF8Block;
        const CUtensorMap* map = big ? &amap128 : &amap;
        if (elect_one()) {
          uint32_t slot = g % kStages, ph = ((g / kStages) & 1u) ^ 1u, i = g;
          for (int kb = kb0; kb < kb1; ++kb, ++i, wp += wbytes) {
            if (!(ok = mbar_wait(&empty[slot], ph, abort_flag, a.err))) break;
            const uint32_t bar = full0 + 8 * slot, sb = base0 + slot * kStageBytes;
            const bool early = kMode != kGateUp && i < pre;
            mbar_arrive_expect_tx_u32(bar, (early ? 0 : wbytes) + abytes);
            if (!early) bulk_load_u32(sb, wp, wbytes, bar, pol_w);
            if (kMode != kGateUp)
              for (int b = 0; b < nbox; ++b)
                tma_load_2d_u32(sb + kBBytes + b * box * kF8Block, map, bar, kb * kF8Block, un.row_start + box * b, pol_act);
            if (++slot == kStages) slot = 0, ph ^= 1u;
          }
        }
        g += kb1 - kb0;
        ok = __all_sync(0xffffffffu, ok);
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer ----------------
      // One elected lane runs a unit's whole K loop: it waits, issues a block's four MMAs and commits.
      // Its own instructions set the pace of a deep K loop (measured in a loop that voted and
      // computed descriptors per MMA: a vote 32 cycles, a barrier probe 46, an MMA 57), so the
      // warp votes once per unit, slots and phases advance incrementally, and the next stage's
      // barrier is probed right after this one's commits.
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty), accf0 = smem_u32(acc_full);
      const uint64_t b0 = smem_desc_sw128(smem_u32(smem));
      uint32_t g = 0;
      bool ok = true;
      for (uint32_t j = 0; ok; ++j) {
        const Unit un = ring.get(j);
        if (un.rows == 0) break;
        ring.done(j);
        const uint32_t idesc = idesc_e4m3_f32(BM, 128u * min(2, a.halves - 2 * un.tile));
        if (elect_one()) {
          uint32_t slot = g % kStages, ph = (g / kStages) & 1u, buf = g & 1u, aph = ((g >> 1) & 1u) ^ 1u;
          bool ready = false;
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!ready && !(ok = mbar_wait(&full[slot], ph, abort_flag, a.err))) break;
            if (!(ok = mbar_wait(&acc_empty[buf], aph, abort_flag, a.err))) break;
            tc_fence_after();
            const uint64_t bdesc = b0 + slot * (kStageBytes >> 4);
            mma_f8_block(tmem + buf * kAccCols, bdesc + (kBBytes >> 4), bdesc, idesc);
            mma_commit_u32(empty0 + 8 * slot);
            mma_commit_u32(accf0 + 8 * buf);
            if (++slot == kStages) slot = 0, ph ^= 1u;
            aph ^= buf;  // both buffers used: their next phase
            buf ^= 1u;
            ready = mbar_test_u32(full0 + 8 * slot, ph);
          }
        }
        g += kb1 - kb0;
        ok = __all_sync(0xffffffffu, ok);
      }
      // all MMAs issued by this warp have finished once `drain` completes
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait_warp(drain, 0, nullptr, a.err);
    } else if (warp == 2) {
      // ---------------- unit list ----------------
      const int total_units = tiles * (kMode >= kLinear ? (a.T + BM - 1) / BM : __ldcg(a.n_segs));
      uint32_t j = 0;
      for (int step = 0;; ++step, ++j) {
        int u;
        if (kMode == kSplit)
          u = step == 0 ? static_cast<int>(blockIdx.x) / a.splits : total_units;
        else if (kMode == kLinear)
          u = blockIdx.x + step * gridDim.x;
        else
          u = mixed_unit(step, total_units);
        const bool more = u < total_units;
        const Unit un = more ? decode_unit<kMode>(u, a, tiles) : Unit{0, 0, 0, 0};
        const int slot = j % kRing;
        if (!mbar_wait_warp(&ring_empty[slot], ((j / kRing) & 1u) ^ 1u, abort_flag, a.err)) break;
        if (kMode == kGateUp)
          for (int n = lane; n < un.rows; n += 32) tok_tab[BM * slot + n] = a.perm[un.row_start + n] / a.k;
        if (lane == 0) ring_rec[slot] = make_int4(un.expert, un.row_start, un.rows, un.tile);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring_full[slot]);
        if (!more) break;
      }
    } else {
      // ---------------- scales ----------------
      // Lane l copies the scales of rows l + 32 i of the tile; a lane's arrival on a group's barrier
      // comes with its copies.
      uint32_t c = 0;
      bool ok = true;
      for (uint32_t j = 0; ok; ++j) {
        const Unit un = ring.get(j);
        if (un.rows == 0) break;
        const float* row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = min(lane + 32 * i, un.rows - 1);
          row[i] = a.as + (kMode == kGateUp ? tok_tab[BM * (j % kRing) + rr] : un.row_start + rr) * a.lds;
        }
        ring.done(j);
        const float* sw = a.ws + (static_cast<int64_t>(un.expert) * tiles + un.tile) * f8_scale_ld(nk) * 2 + 4 * (lane & 1);
        for (int gi = kb0 / 4; 4 * gi < kb1; ++gi, ++c) {
          const int slot = c % kScGroups;
          if (!(ok = mbar_wait_warp(&sc_empty[slot], ((c / kScGroups) & 1u) ^ 1u, abort_flag, a.err))) break;
          const uint32_t dst = smem_u32(sc_tab + slot * kScGroupBytes);
          const uint32_t bytes = 4u * min(4, nk - 4 * gi);  // a row may end with its last block's scale
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (32 * i < un.rows) cp_async_16_part(dst + (lane + 32 * i) * 16, row[i] + 4 * gi, bytes);
          if (lane < 2) cp_async_16(dst + BM * 16 + 16 * lane, sw + 8 * gi);
          cp_async_arrive(&sc_full[slot]);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();  // none is in flight when the CTA ends
    }
  } else if (warp < kFirstGather) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg<kMode>::kRegsEpi));
    // ---------------- epilogue ----------------
    const int q = warp & 3, half = (warp - kFirstEpi) >> 2;
    const int r = 32 * q + lane;  // row of the tile
    const uint32_t stage_out = smem_u32(out_tab + (warp - kFirstEpi) * (kMode == kLinear ? kTmaOutBytes : kOutBytes));
    // y is read back by the next launch: keep it in L2 ahead of the streamed weights
    const uint64_t pol_out = kMode == kDown ? l2_policy_evict_last() : l2_policy_evict_first();
    uint32_t g = 0, c = 0, nx = 0;  // K blocks, groups of scales, exchanges of row maxima so far
    bool ok = true;
    const uint32_t accf0 = smem_u32(acc_full), acce0 = smem_u32(acc_empty);
    const uint32_t tacc = tmem + (static_cast<uint32_t>(32 * q) << 16) + half * 128;
    uint32_t limit = kSpinLimit;
    auto spin = [&](uint32_t bar, uint32_t parity) {
      uint32_t n = 0;
      while (!__all_sync(0xffffffffu, mbar_try_wait_u32(bar, parity)))
        if (++n >= limit) {
          limit = 0;
          break;
        }
    };
    for (uint32_t j = 0; ok; ++j) {
      const Unit un = ring.get(j);
      if (un.rows == 0) break;
      ring.done(j);
      const bool on = 32 * q < un.rows && half < a.halves - 2 * un.tile;  // some row and column is wanted
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      // The loop over K blocks is kept short, its waits included: its time follows its length in
      // instructions (unrolled by two, the 8192-row product of an earlier form, 133 us, took 228).  A wait is a
      // bounded spin of the whole warp; one that gives up leaves limit 0, and the warp goes on without
      // waiting to the end of the unit, where it reports.
      int kb = kb0;
      if (!on) {
        for (; kb < kb1; ++kb, ++g) {
          spin(accf0 + 8 * (g & 1u), (g >> 1) & 1u);
          mbar_arrive_lane0(&acc_empty[g & 1u]);
          if ((kb & 3) == 3 || kb == kb1 - 1) mbar_arrive_lane0(&sc_empty[c++ % kScGroups]);
        }
      }
      uint32_t buf = g & 1u, ph = (g >> 1) & 1u;
#pragma unroll 1
      while (kb < kb1) {  // a group of scales
        const uint32_t slot = c % kScGroups;
        spin(smem_u32(&sc_full[slot]), (c / kScGroups) & 1u);
        const uint32_t grp = smem_u32(sc_tab + slot * kScGroupBytes);
        uint32_t pa = grp + 16 * r + 4 * (kb & 3), pw = grp + 16 * BM + 8 * (kb & 3);
        const int end = min((kb | 3) + 1, kb1);
        g += end - kb;
#pragma unroll 1
        for (; kb < end; ++kb, pa += 4, pw += 8) {
          const float sa = ld_shared_f32(pa);
          const float2 w = ld_shared_v2(pw);
          spin(accf0 + 8 * buf, ph);
          tc_fence_after();
          const float s0 = sa * (kMode == kGateUp || half == 0 ? w.x : w.y);
          const float s1 = kMode == kGateUp ? sa * w.y : s0;
          add_block(acc, tacc + buf * kAccCols, pack_f32x2(s0, s0), pack_f32x2(s1, s1), acce0 + 8 * buf);
          ph ^= buf;  // both buffers used: their next phase
          buf ^= 1u;
        }
        mbar_arrive_lane0(&sc_empty[slot]);  // (every lane has read the group's scales)
        ++c;
      }
      if (limit == 0) {
        set_error(a.err, MOE_DEVERR_TIMEOUT);
        *abort_flag = 1;
        ok = false;
      }
      if (!ok) break;
      const int64_t grow = un.row_start + r;
      if (kMode == kGateUp) {
        // columns 0..63 gate, 64..127 up of features 64 half .. + 63 of the tile's 128
        float h[64], amax = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float g0, g1, u0, u1;
          unpack_f32x2(acc[i], g0, g1);
          unpack_f32x2(acc[32 + i], u0, u1);
          h[2 * i] = swiglu(g0, u0);
          h[2 * i + 1] = swiglu(g1, u1);
          amax = fmaxf(amax, fmaxf(fabsf(h[2 * i]), fabsf(h[2 * i + 1])));
        }
        // the block's scale needs the other half's maximum (the lane quarter's two warps make the same
        // exchanges); slots alternate: one is written again only after its reader arrived in between
        const int slot = (nx & 1) * 2 * BM;
        xch[slot + half * BM + r] = amax;
        __syncwarp();
        if (lane == 0) mbar_arrive(&xch_bar[q]);
        if (!(ok = mbar_wait_warp(&xch_bar[q], nx & 1u, abort_flag, a.err))) break;
        ++nx;
        amax = fmaxf(amax, xch[slot + (half ^ 1) * BM + r]);
        const float sc = f8_scale(amax);
        const float rs = __frcp_rn(sc);
        if (r < un.rows) {
          uint8_t* o = a.hq + grow * a.ldh + un.tile * 128 + half * 64;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float* v = h + 32 * c + 4 * i;
              w[i] = f32x2_to_e4m3x2(v[0] * rs, v[1] * rs) | (f32x2_to_e4m3x2(v[2] * rs, v[3] * rs) << 16);
            }
            st_global_v8(o + 32 * c, w);
          }
          if (half == 0) a.hs[grow * a.ldhs + un.tile] = sc;
        }
      } else if (kMode == kSplit) {
        if (r < un.rows) {  // (every MMA of this CTA has read its operands: the stages are free)
          const uint32_t mine = smem_u32(smem) + r * kSumPitch + half * 512;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            st_shared_v4(mine + 16 * c, static_cast<uint32_t>(acc[2 * c]), static_cast<uint32_t>(acc[2 * c] >> 32),
                         static_cast<uint32_t>(acc[2 * c + 1]), static_cast<uint32_t>(acc[2 * c + 1] >> 32));
        }
      } else {
        store_rows<kMode>(acc, a, &omap, stage_out, un.row_start + 32 * q, un.rows - 32 * q, un.tile * 256 + half * 128, pol_out);
      }
    }
    if (kMode == kLinear && lane == 0) bulk_wait_all();  // the stores are done before the CTA is
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg<kMode>::kRegsRest));
    // ---------------- gate/up: row gather (cp.async) ----------------
    // Warp w owns stage slot w: it fills every stage g with g % kStages == w, waits for its own copies, fences
    // them for the tensor core and arrives.  8 consecutive lanes copy one row's 128 bytes; the addresses of 8
    // rows a lane are formed before their copies, so that the reads of the row table overlap.  (One row
    // after the other: Zipf layer 460 us instead of 452.  A quarter of each stage a warp, announced two stages
    // later: 452, but 2% more for a decode step.  TMA gathers of four rows, about 85 cycles each: 587.)
    const int slot = warp - kFirstGather;
    const int ch = lane & 7, nl = lane >> 3;
    const uint32_t d0 = smem_u32(smem + slot * kStageBytes + kBBytes) + nl * 128;
    const uint32_t dx[2] = {d0 + ((ch ^ nl) << 4), d0 + ((ch ^ (nl + 4)) << 4)};
    const uint64_t pol_x = l2_policy_evict_last();
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t j = 0; ok; ++j) {
      const Unit un = ring.get(j);
      if (un.rows == 0) break;
      const int32_t* tok = tok_tab + BM * (j % kRing);
      for (int kb = kb0; kb < kb1; ++kb, ++g) {
        if (static_cast<int>(g % kStages) != slot) continue;
        if (!(ok = mbar_wait_warp(&empty[slot], ((g / kStages) & 1u) ^ 1u, abort_flag, a.err))) break;
        const uint8_t* base = a.a + kb * kF8Block + ch * 16;
        for (int n = nl; n < un.rows; n += 4 * 8) {
          const uint8_t* src[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) src[i] = base + static_cast<size_t>(tok[min(n + 4 * i, un.rows - 1)]) * a.lda;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n + 4 * i < un.rows) cp_async_16_hint(dx[i & 1] + (n - nl + 4 * i) * 128, src[i], pol_x);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_lane0(&full[slot]);
      }
      ring.done(j);
    }
  }

  if (kMode == kSplit) {
    // every thread of the cluster meets; then each CTA adds up its share of the columns
    __syncthreads();
    cluster_sync();
    const int u = static_cast<int>(blockIdx.x) / a.splits;
    const Unit un = decode_unit<kMode>(u, a, tiles);
    const int cols = min(256, a.N - 256 * un.tile), per = 256 / a.splits;
    const int c0 = split * per, quads = per / 4;
    for (int i = threadIdx.x; i < un.rows * quads; i += Cfg<kMode>::kThreads) {
      const int row = i / quads, c = c0 + 4 * (i % quads);
      if (c >= cols) continue;
      const uint32_t at = smem_u32(smem) + row * kSumPitch + 4 * c;
      float4 v = ld_cluster_v4(at, 0);
      for (int p = 1; p < a.splits; ++p) {
        const float4 w = ld_cluster_v4(at, p);
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
      }
      const int64_t o = (un.row_start + row) * a.ldo + 256 * un.tile + c;
      const float f[4] = {v.x, v.y, v.z, v.w};
      if (a.out_type == MOE_BF16) {
        uint16_t* out = static_cast<uint16_t*>(a.out) + o;
        if (a.out_vec && c + 4 <= cols)
          *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
        else
          for (int k = 0; k < 4 && c + k < cols; ++k) out[k] = f32_to_bf16_bits_rn(f[k]);
      } else {
        float* out = static_cast<float*>(a.out) + o;
        if (a.out_vec && c + 4 <= cols)
          *reinterpret_cast<float4*>(out) = v;
        else
          for (int k = 0; k < 4 && c + k < cols; ++k) out[k] = f[k];
      }
    }
    cluster_sync();  // no CTA leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  abort_quiesce(abort_flag);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace f8

template <int kMode>
static cudaError_t launch_f8(const CUtensorMap& m, const CUtensorMap& m128, const CUtensorMap& o, const F8Args& a,
                             int num_sms, cudaStream_t st) {
  auto kern = f8::f8_gemm_kernel<kMode>;
  cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), f8::Cfg<kMode>::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(num_sms), dim3(f8::Cfg<kMode>::kThreads), f8::Cfg<kMode>::kSmemBytes, st, m, m128, o, a);
}

cudaError_t launch_f8_gateup(const F8Args& a, int num_sms, cudaStream_t st) {
  return launch_f8<f8::kGateUp>(CUtensorMap{}, CUtensorMap{}, CUtensorMap{}, a, num_sms, st);
}
cudaError_t launch_f8_down(const CUtensorMap* amap, const CUtensorMap* amap128, const F8Args& a, int num_sms,
                           cudaStream_t st) {
  return launch_f8<f8::kDown>(*amap, *amap128, CUtensorMap{}, a, num_sms, st);
}

// Clusters of `s` CTAs of the split kernel that the device runs at the same time (0: unknown).
static int split_clusters(int s) {
  static std::mutex mu;
  static std::map<std::pair<int, int>, int> known;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(mu);
  auto it = known.find({dev, s});
  if (it != known.end()) return it->second;
  using C = f8::Cfg<f8::kSplit>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(s), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, f8::f8_gemm_kernel<f8::kSplit>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  try {
    known[{dev, s}] = n;
  } catch (...) {  // no memory for the note: the next call asks again
  }
  return n;
}

// Units too few to fill the SMs (small T, or a small matrix) are split along K over clusters of 8, 4 or
// 2 CTAs: as many as run at the same time with a K block or more each.
cudaError_t launch_f8_linear(const CUtensorMap* amap, const CUtensorMap* omap, const F8Args& a, int num_sms,
                             cudaStream_t st) {
  const int units = (a.halves + 1) / 2 * ((a.T + f8::BM - 1) / f8::BM);
  if (2 * units <= num_sms && a.nk >= 2) {
    auto kern = f8::f8_gemm_kernel<f8::kSplit>;
    using C = f8::Cfg<f8::kSplit>;
    cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::kSmemBytes);
    if (e != cudaSuccess) return e;
    for (int s = 8; s >= 2; s /= 2) {
      if (s > a.nk || units * s > num_sms || units > split_clusters(s)) continue;
      F8Args b = a;
      b.splits = s;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(units * s);
      cfg.blockDim = dim3(C::kThreads);
      cfg.dynamicSmemBytes = C::kSmemBytes;
      cfg.stream = st;
      cudaLaunchAttribute attr[2];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim = {static_cast<unsigned>(s), 1, 1};
      cfg.attrs = attr;
      cfg.numAttrs = 2;
      return cudaLaunchKernelEx(&cfg, kern, *amap, CUtensorMap{}, CUtensorMap{}, b);
    }
  }
  return launch_f8<f8::kLinear>(*amap, CUtensorMap{}, *omap, a, units < num_sms ? units : num_sms, st);
}

}  // namespace moe
