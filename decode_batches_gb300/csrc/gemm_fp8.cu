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
// Three uses of one kernel:
//   gate/up  a = rows of x gathered by the permutation; a tile's 256 weight rows are two times (64
//            gate rows, the same 64 features' up rows); the epilogue forms silu(g) * u in fp32,
//            quantises the 128 features (one activation block of h) and writes codes and scale.
//   down     a = those rows of h; y in fp16 in grouped order for the combine.
//   linear   a = the T rows of one matrix; bf16 or fp32 out.
// Routed units are ordered tile-major within an expert's parts, linear units tile-major over the
// row parts: CTAs that share a weight tile run side by side and its second read is served by L2.
//
// Roles (persistent CTAs, one per SM, every role walks the same unit sequence):
//   warp 0      producer: weights by bulk copy (tile-contiguous, pre-swizzled); rows by TMA
//   warp 1      TMEM owner and MMA issuer
//   warps 4-11  epilogue: warps 4-7 the tile's first half, 8-11 the second; TMEM lanes 32 (warp % 4)
//   warps 12-15 gate/up: cp.async gather of the rows, one warp per stage slot
// Registers move from the first (and the gather) warps to the epilogue warps, which hold 128 sums a
// thread.  TMEM: two buffers of 256 columns, so one block's MMAs overlap the previous block's sums.
// Rows of a tile beyond the segment's are never copied: whatever the slot held lands in lanes that
// nobody reads.
#include "fp8.cuh"
#include "kernels.h"

namespace moe {
namespace f8 {

constexpr int kGateUp = 0, kDown = 1, kLinear = 2;
constexpr int BM = 128;                           // activation rows per tile (MMA M)
constexpr int kStages = 4;
constexpr int kBBytes = 2 * kF8TileBytes;         // 256 weight rows x 128 K elements
constexpr int kABytes = BM * kF8Block;
constexpr int kStageBytes = kABytes + kBBytes;    // 48 KB
constexpr int kAccCols = 256;
constexpr int kTmemCols = 2 * kAccCols;
constexpr int kEpiWarps = 8, kFirstEpi = 4, kFirstGather = 12;
constexpr int kTokBytes = kStages * BM * 4;       // per gather warp: source row of each row
constexpr int kXchBytes = 2 * 2 * BM * 4;         // row maxima of h: [unit parity][half][row]
constexpr int kSmemBytes = kStages * kStageBytes + 1024 /*barriers*/ + 1024 /*align slack*/ + kTokBytes + kXchBytes;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

template <int kMode>
struct Cfg {
  static constexpr int kThreads = kMode == kGateUp ? 512 : 384;
  // register split: the sums over the warpgroups equal the launch's (128 x 4 or 168 x 3)
  static constexpr int kRegsEpi = kMode == kGateUp ? 208 : 216;
  static constexpr int kRegsRest = kMode == kGateUp ? 48 : 72;
};

struct Unit {
  int expert, row_start, rows, tile, ntile;  // ntile: halves of the tile (1 or 2)
};

MOE_DEVICE Seg load_seg(const Seg* p) {  // through L2: the down kernel's producer reads them before its wait
  const int4 lo = __ldcg(reinterpret_cast<const int4*>(p));
  const int4 hi = __ldcg(reinterpret_cast<const int4*>(p) + 1);
  return Seg{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

template <int kMode>
MOE_DEVICE Unit decode_unit(int u, const F8Args& a, int tiles) {
  Unit un;
  if (kMode == kLinear) {
    const int parts = (a.T + BM - 1) / BM;
    const int p = u % parts, q = a.T / parts, rem = a.T % parts;
    un.expert = 0;
    un.tile = u / parts;
    un.row_start = p * q + min(p, rem);
    un.rows = q + (p < rem ? 1 : 0);
  } else {
    const Seg any = load_seg(a.segs + u / tiles);
    const int o = u - any.first * tiles;
    const Seg s = load_seg(a.segs + any.first + o % any.nparts);
    un.expert = s.expert;
    un.tile = o / any.nparts;
    un.row_start = s.row_start;
    un.rows = s.rows;
  }
  un.ntile = min(2, a.halves - 2 * un.tile);
  return un;
}

// Adds 128 columns of one K block, times the scales (s01 the first 64 columns', s23 the rest's), to
// the thread's sums: 16-column loads, one in flight while the previous one is added.
MOE_DEVICE void add_block(uint64_t (&acc)[64], uint32_t taddr, uint64_t s01, uint64_t s23) {
  uint32_t r[2][16];
  tmem_ld_32x32b_x16(taddr, r[0]);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    tmem_wait_ld16(r[c & 1]);
    if (c < 7) tmem_ld_32x32b_x16(taddr + 16 * (c + 1), r[(c + 1) & 1]);
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

// One row's 128 columns (col0 .. of N) of type out_type.
template <int kMode>
MOE_DEVICE void store_row(const uint64_t (&acc)[64], const F8Args& a, int64_t row, int col0) {
  const int n = a.N - col0;  // valid columns here
  if (kMode == kDown || a.out_type == MOE_FP16) {
    uint16_t* o = static_cast<uint16_t*>(a.out) + row * a.ldo + col0;
    bool sat = false;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float lo, hi;
        unpack_f32x2(acc[8 * c + i], lo, hi);
        if (fabsf(lo) > kF16Max || lo != lo) sat |= 16 * c + 2 * i < n, lo = lo != lo ? lo : copysignf(kF16Max, lo);
        if (fabsf(hi) > kF16Max || hi != hi) sat |= 16 * c + 2 * i + 1 < n, hi = hi != hi ? hi : copysignf(kF16Max, hi);
        w[i] = static_cast<uint32_t>(f32_to_f16_bits_rn(lo)) | (static_cast<uint32_t>(f32_to_f16_bits_rn(hi)) << 16);
      }
      if (a.out_vec && 16 * c + 16 <= n) {
        st_global_v8(o + 16 * c, w);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (16 * c + i < n) o[16 * c + i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
      }
    }
    if (sat) set_error(a.err, MOE_DEVERR_RANGE);
  } else if (a.out_type == MOE_BF16) {
    uint16_t* o = static_cast<uint16_t*>(a.out) + row * a.ldo + col0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float lo, hi;
        unpack_f32x2(acc[8 * c + i], lo, hi);
        w[i] = pack_bf16x2(lo, hi);
      }
      if (a.out_vec && 16 * c + 16 <= n) {
        st_global_v8(o + 16 * c, w);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (16 * c + i < n) o[16 * c + i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
      }
    }
  } else {
    float* o = static_cast<float*>(a.out) + row * a.ldo + col0;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack_f32x2(acc[4 * c + i], lo, hi);
        w[2 * i] = __float_as_uint(lo), w[2 * i + 1] = __float_as_uint(hi);
      }
      if (a.out_vec && 8 * c + 8 <= n) {
        st_global_v8(o + 8 * c, w);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * c + i < n) o[8 * c + i] = __uint_as_float(w[i]);
      }
    }
  }
}

template <int kMode>
__global__ void __launch_bounds__(Cfg<kMode>::kThreads, 1)
    f8_gemm_kernel(const __grid_constant__ CUtensorMap amap, const F8Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* xch_bar = acc_empty + 2;   // per lane quarter: both halves published their row maxima
  uint64_t* drain = xch_bar + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* tok_tab = reinterpret_cast<int32_t*>(smem + kStages * kStageBytes + 1024);
  volatile float* xch = reinterpret_cast<volatile float*>(smem + kStages * kStageBytes + 1024 + kTokBytes);

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
    if (warp != 0) pdl_wait();
  }

  const int tiles = (a.halves + 1) / 2;
  const int nk = a.nk;
  const int total_units = tiles * (kMode == kLinear ? (a.T + BM - 1) / BM : __ldcg(a.n_segs));

  if (warp < kFirstEpi) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg<kMode>::kRegsRest));
    if (warp == 0) {
      // ---------------- producer ----------------
      const uint64_t pol_w = l2_policy_evict_first();
      const uint64_t pol_act = l2_policy_evict_last();
      uint32_t pre = 0;  // stages whose weights were requested before the dependency wait
      if (kMode != kGateUp) {
        for (int u = blockIdx.x; u < total_units && pre < static_cast<uint32_t>(kStages); u += gridDim.x) {
          const Unit un = decode_unit<kMode>(u, a, tiles);
          const uint8_t* wb = a.w + un.expert * a.w_stride;
          for (int kb = 0; kb < nk && pre < static_cast<uint32_t>(kStages); ++kb, ++pre) {
            if (elect_one()) {  // a fresh slot: no wait; the arrival comes with the rows below
              mbar_expect_tx(&full[pre], un.ntile * kF8TileBytes);
              bulk_load(smem + pre * kStageBytes, wb + f8_half_offset(2 * un.tile, kb, a.halves, nk),
                        un.ntile * kF8TileBytes, &full[pre], pol_w);
            }
            __syncwarp();
          }
        }
        pdl_wait();
      }
      uint32_t g = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
        const Unit un = decode_unit<kMode>(u, a, tiles);
        const uint8_t* wb = a.w + un.expert * a.w_stride;
        const int nbox = kMode == kGateUp ? 0 : (un.rows + 31) / 32;
        for (int kb = 0; kb < nk; ++kb, ++g) {
          const int slot = g % kStages;
          if (!(ok = mbar_wait_warp(&empty[slot], ((g / kStages) & 1u) ^ 1u, abort_flag, a.err))) break;
          if (elect_one()) {
            uint8_t* sb = smem + slot * kStageBytes;
            const bool early = g < pre;
            mbar_arrive_expect_tx(&full[slot], (early ? 0 : un.ntile * kF8TileBytes) + nbox * 32 * kF8Block);
            if (!early)
              bulk_load(sb, wb + f8_half_offset(2 * un.tile, kb, a.halves, nk), un.ntile * kF8TileBytes, &full[slot],
                        pol_w);
            if (kMode != kGateUp)
              for (int i = 0; i < nbox; ++i)
                tma_load_2d(sb + kBBytes + i * 32 * kF8Block, &amap, &full[slot], kb * kF8Block, un.row_start + 32 * i,
                            pol_act);
          }
          __syncwarp();
        }
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer: the warp waits, one elected lane issues ----------------
      uint32_t g = 0;
      bool ok = true, ready = false;  // ready: full[g % kStages] already seen complete for stage g
      for (int u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
        const Unit un = decode_unit<kMode>(u, a, tiles);
        const uint32_t idesc = idesc_e4m3_f32(BM, 128u * un.ntile);
        for (int kb = 0; kb < nk; ++kb, ++g) {
          const int slot = g % kStages;
          const uint32_t buf = g & 1u, use_acc = g >> 1;
          if (!ready && !(ok = mbar_wait_warp(&full[slot], (g / kStages) & 1u, abort_flag, a.err))) break;
          if (!(ok = mbar_wait_warp(&acc_empty[buf], (use_acc & 1u) ^ 1u, abort_flag, a.err))) break;
          const uint32_t gn = g + 1;  // probe the next stage now, use the answer next iteration
          const bool next = mbar_test(&full[gn % kStages], (gn / kStages) & 1u);
          tc_fence_after();
          const uint32_t sb = smem_u32(smem + slot * kStageBytes);
          const uint64_t bdesc = smem_desc_sw128(sb);
          const uint64_t adesc = smem_desc_sw128(sb + kBBytes);
          const uint32_t d_tmem = tmem + buf * kAccCols;
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < kF8Block / 32; ++ks)  // K = 32 per MMA: +32 bytes = +2 in the address field
              mma_f8_ss(d_tmem, adesc + 2 * ks, bdesc + 2 * ks, idesc, ks != 0);
            mma_commit(&empty[slot]);
            mma_commit(&acc_full[buf]);
          }
          __syncwarp();
          ready = __all_sync(0xffffffffu, next);
        }
      }
      // all MMAs issued by this warp have finished once `drain` completes
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait_warp(drain, 0, nullptr, a.err);
    }
  } else if (warp < kFirstGather) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg<kMode>::kRegsEpi));
    // ---------------- epilogue ----------------
    const int q = warp & 3, half = (warp - kFirstEpi) >> 2;
    const int r = 32 * q + lane;  // row of the tile
    uint32_t g = 0, nx = 0;  // nx: exchanges of row maxima so far
    bool ok = true;
    for (int u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
      const Unit un = decode_unit<kMode>(u, a, tiles);
      const bool on = 32 * q < un.rows && half < un.ntile;  // warp-uniform: some row and column is wanted
      const int64_t grow = un.row_start + min(r, un.rows - 1);
      int64_t srow = grow;
      if (kMode == kGateUp) srow = a.perm[grow] / a.k;
      const float4* sa4 = reinterpret_cast<const float4*>(a.as + srow * a.lds);
      const float2* sw = reinterpret_cast<const float2*>(a.ws) + (static_cast<int64_t>(un.expert) * tiles + un.tile) * nk;
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      float4 sa_now = make_float4(0.f, 0.f, 0.f, 0.f), sa_next = sa_now;
      float2 sw_next = make_float2(0.f, 0.f);
      if (on) {
        sa_next = sa4[0];
        sw_next = __ldg(sw);
      }
      for (int kb = 0; kb < nk; ++kb, ++g) {
        const uint32_t buf = g & 1u, use_acc = g >> 1;
        const float2 w2 = sw_next;
        if (on) {  // the next blocks' scales are requested a block (four blocks) ahead
          if ((kb & 3) == 0) {
            sa_now = sa_next;
            if (kb + 4 < nk) sa_next = sa4[(kb >> 2) + 1];
          }
          if (kb + 1 < nk) sw_next = __ldg(sw + kb + 1);
        }
        const float sa = (kb & 2) ? ((kb & 1) ? sa_now.w : sa_now.z) : ((kb & 1) ? sa_now.y : sa_now.x);
        if (!(ok = mbar_wait_warp(&acc_full[buf], use_acc & 1u, abort_flag, a.err))) break;
        if (on) {
          tc_fence_after();
          const float s0 = kMode == kGateUp ? sa * w2.x : sa * (half ? w2.y : w2.x);
          const float s1 = kMode == kGateUp ? sa * w2.y : s0;
          add_block(acc, tmem + (static_cast<uint32_t>(32 * q) << 16) + buf * kAccCols + half * 128, pack_f32x2(s0, s0),
                    pack_f32x2(s1, s1));
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
      }
      if (!ok) break;
      if (!on) continue;
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
      } else {
        if (r < un.rows) store_row<kMode>(acc, a, grow, un.tile * 256 + half * 128);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg<kMode>::kRegsRest));
    // ---------------- gate/up: row gather (cp.async) ----------------
    // Warp w owns stage slot w: it fills every stage g with g % kStages == w, waits for its own
    // copies, fences them for the tensor core and arrives.  8 consecutive lanes copy one row's
    // 128 bytes.
    const int slot = warp - kFirstGather;
    int32_t* tok = tok_tab + BM * slot;
    const int ch = lane & 7;
    const uint64_t pol_x = l2_policy_evict_last();
    uint32_t g = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
      const Unit un = decode_unit<kMode>(u, a, tiles);
      bool have_tok = false;
      for (int kb = 0; kb < nk; ++kb, ++g) {
        const int s = g % kStages;
        if (s != slot) continue;
        if (!have_tok) {
          for (int n = lane; n < un.rows; n += 32) tok[n] = a.perm[un.row_start + n] / a.k;
          __syncwarp();
          have_tok = true;
        }
        if (!(ok = mbar_wait_warp(&empty[s], ((g / kStages) & 1u) ^ 1u, abort_flag, a.err))) break;
        const uint32_t sa = smem_u32(smem + s * kStageBytes + kBBytes);
        const int k0 = kb * kF8Block + ch * 16;
        for (int n = lane >> 3; n < un.rows; n += 4)
          cp_async_16_hint(sa + n * 128 + ((ch ^ (n & 7)) << 4), a.a + static_cast<size_t>(tok[n]) * a.lda + k0, pol_x);
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
      __syncwarp();  // the table is read by the whole warp before the next unit rewrites it
    }
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
static cudaError_t launch_f8(const CUtensorMap& m, const F8Args& a, int num_sms, cudaStream_t st) {
  auto kern = f8::f8_gemm_kernel<kMode>;
  cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), f8::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(num_sms), dim3(f8::Cfg<kMode>::kThreads), f8::kSmemBytes, st, m, a);
}

cudaError_t launch_f8_gateup(const F8Args& a, int num_sms, cudaStream_t st) {
  return launch_f8<f8::kGateUp>(CUtensorMap{}, a, num_sms, st);
}
cudaError_t launch_f8_down(const CUtensorMap* amap, const F8Args& a, int num_sms, cudaStream_t st) {
  return launch_f8<f8::kDown>(*amap, a, num_sms, st);
}
cudaError_t launch_f8_linear(const CUtensorMap* amap, const F8Args& a, int num_sms, cudaStream_t st) {
  const int units = (a.halves + 1) / 2 * ((a.T + f8::BM - 1) / f8::BM);
  return launch_f8<f8::kLinear>(*amap, a, units < num_sms ? units : num_sms, st);
}

}  // namespace moe
