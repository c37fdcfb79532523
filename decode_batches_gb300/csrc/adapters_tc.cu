// Low-rank adapters of larger steps on the tensor cores (adapters.cu has the formulas and the small steps' kernel).
//
// A tile is up to 128 rows of one adapter, a cluster of C CTAs computes it:
//   shrink  D[rows][R] = x A^T over this CTA's range of K: tcgen05 MMAs of 128 (or 64) x R x 16, rows of x gathered with
//           cp.async into the 128-byte-swizzled operand, A in tiles packed that way (bulk copies), a ring of 64-column
//           stages;
//   u       the CTAs' partial sums meet in distributed shared memory: each CTA adds up its share of the rows, scales and
//           splits them into two or three 16-bit terms (adapter_split) and writes those into every CTA's MMA operand;
//   expand  128 features at a time, over this CTA's range of N: D[rows][128] = (sum of the terms) B^T, an MMA a term and
//           16 ranks, D double buffered in TMEM; W warps add the base and write.
// Bound by memory: x, base and out pass once; the weights are read once a tile, from L2, whose way to an SM is as tight
// (64 bytes a ns and SM in either phase): so tiles are as large as still leave every SM one.  8195 rows of 4096 x 4096 in
// 32 adapters of rank 64: 52 us, of which 12 the gather (83 MB), 23 the expand (150 MB), 6 u's way through the cluster, 9
// the grouping's launch and the two starts; the floor is 33.  Warp-level fragments in the small steps' manner took 85 us
// and 24 M instructions there (14 M here).
//
// The rows of a B tile are permuted within 32 features such that the 16x256b TMEM load hands a lane eight neighbouring
// features of a row: base and out move as 16-byte vectors, 64 contiguous bytes a row, without a transposition.
#include "adapters.cuh"
#include "adapters_split.cuh"
#include "cluster.cuh"
#include "elems.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;             // rows of a tile at most (the MMA's M; 64 where all tiles have that many at most)
constexpr int kSlice = 128;            // features of an expand step
constexpr int kStagesMax = 8;

// Shared memory: the ring, then u.  During the shrink its stages run on into u's place; after it the ring's start holds
// the partial sums, B's first tiles come behind them and the later ones, once the sums are read, also in their place.
template <int R, int W, bool kFp16>
struct Cfg {
  static constexpr int kThreads = 32 * (W + 1);      // W warps gather, add up and write, one lane issues
  static constexpr int kCtas = W == 8 ? 2 : 1;       // an SM
  static constexpr int kWBytes = R * 128;
  static constexpr int kTerm = kRows * R * 2;        // one of u's terms
  static constexpr int kU = kAdapterTerms<kFp16> * kTerm;
  static constexpr int kPart = kRows * R * 4;        // partial sums
  static constexpr int kBTile = kSlice * R * 2;
  // (a third term takes its place from the ring, which the stages run on out of: with more shared memory in all, less L1 was
  // left for the base's lines, 8195 fp32 rows 84 us instead of 71)
  static constexpr int kRing = (W == 8 ? 72 : R <= 64 ? 160 : 128) * 1024 - (kU - 2 * kTerm);
  static constexpr int kBEarly = (kRing - kPart) / kBTile < 4 ? (kRing - kPart) / kBTile : 4;
  static constexpr int kBSlots = kBEarly + kPart / kBTile;
  static_assert(W == 16 || (W == 8 && R <= 64), "");
  static constexpr int kRowBytes = (R < 64 ? R : 64) * 2;  // a row of u or of a B tile within a block of 64 ranks
  static constexpr int kTail = kRows * 8 + 320;
  static constexpr int kBytes = kRing + kU + kTail + 1024;
  // The shrink's accumulators, taken in turn by its steps: the tensor core cuts a sum's last bits at every step, always
  // towards zero, and a quarter or an eighth of the steps leaves as little of that (an fp32 result of 8195 rows, K =
  // 4096, two CTAs: 2.3e-6 off the formula with one, 2.9e-7 with eight, and fp32 products 2.4e-7).
  static constexpr int kAccs = W == 8 && R == 64 || R == 128 ? 4 : 8;
  static constexpr int kTmemCols = kAccs * R <= 256 ? 256 : 512;  // (the expand's two buffers are 256)
  static_assert(kCtas * kTmemCols <= 512, "");
  static constexpr int b_at(int slot) { return slot < kBEarly ? kPart + slot * kBTile : (slot - kBEarly) * kBTile; }
  static_assert(kBEarly >= 1 && kBSlots <= 6 && kBytes <= 227 * 1024 && kCtas * (kBytes + 1024) <= 228 * 1024, "");
  // Stages for tiles of `rows` rows (64 or 128): 6 of 16 KB or 4 of 24 at rank 64 with two CTAs an SM.
  static constexpr int stage_bytes(int rows) { return rows * 128 + kWBytes; }
  static constexpr int stages(int rows) {
    const int n = (kRing + kU) / stage_bytes(rows);
    return n < kStagesMax ? n : kStagesMax;
  }
};

// Terms of u that the expand takes: a 16-bit result gets two, whose 2^-17 of the adapter's part lie far below the rounding
// of result and base, 2^-9 or 2^-12 (a third costs 1 us of 52 in the 8195 rows, and 1 of 19 in 200 rows of rank 64).
template <bool kFp16>
MOE_DEVICE int u_terms(const AdapterArgs& p) {
  return p.out_type == MOE_FP32 ? kAdapterTerms<kFp16> : 2;
}

// Byte offset of 16-byte piece p of row r in a tile of kRowBytes-wide rows, swizzled over the row's own width.
template <int kRowBytes>
MOE_DEVICE constexpr uint32_t swizzled(uint32_t r, uint32_t p) {
  const uint32_t at = r * kRowBytes + p * 16;
  return at ^ ((at >> 3) & (kRowBytes - 16u));
}

// Descriptor of a K-major operand of kRowBytes-wide rows with the swizzle of that width: groups of 8 rows are
// 8 kRowBytes apart; layout 2, 4 or 6 (128, 64 or 32 bytes).
template <int kRowBytes>
MOE_DEVICE uint64_t operand_desc(uint32_t addr) {
  constexpr uint64_t layout = kRowBytes == 128 ? 2 : kRowBytes == 64 ? 4 : 6;
  return (static_cast<uint64_t>((addr >> 4) & 0x3FFFu)) | (1ull << 16) | (static_cast<uint64_t>(8 * kRowBytes >> 4) << 32) |
         (1ull << 46) | (layout << 61);
}

// 16 lanes x 32 columns: lane (g, q) gets rows g and g + 8 (of the 16 at taddr's lane), and of each 8 columns i the
// columns 8 i + 2 q, 8 i + 2 q + 1: r[4 i], r[4 i + 1] of row g, r[4 i + 2], r[4 i + 3] of row g + 8.
MOE_DEVICE void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

MOE_DEVICE void st_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
MOE_DEVICE void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// Generic writes (also to another CTA's shared memory) before the tensor core's reads.
MOE_DEVICE void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

template <int R, int W, bool kFp16>
struct Smem {
  uint8_t* ring;
  uint8_t* u;
  int* rows;         // [128] row numbers, -1 past the last
  float* row_scale;  // [128] (fp16)
  uint64_t* full;    // [kStagesMax] the threads that copy x, and A's copy
  uint64_t* empty;   // [kStagesMax]
  uint64_t* b_full;  // [kBSlots]
  uint64_t* b_empty;
  uint64_t* o_full;  // [2] D of an expand step
  uint64_t* o_empty;
  uint64_t* d_full;  // the shrink's D
  int tile_rows;     // 64 or 128: rows that the stages and the MMAs are made for
  int spare;         // rows without an adapter that this cluster copies
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  MOE_DEVICE explicit Smem(uint8_t* raw) {
    uint8_t* p = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    ring = p, p += Cfg<R, W, kFp16>::kRing;
    u = p, p += Cfg<R, W, kFp16>::kU;
    rows = reinterpret_cast<int*>(p), p += kRows * 4;
    row_scale = reinterpret_cast<float*>(p), p += kRows * 4;
    full = reinterpret_cast<uint64_t*>(p);
    empty = full + kStagesMax, b_full = empty + kStagesMax, b_empty = b_full + 6, o_full = b_empty + 6, o_empty = o_full + 2;
    d_full = o_empty + 2;
    tmem_slot = reinterpret_cast<uint32_t*>(d_full + 1);
    abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  }
};

// ---- the issuing lane ----------------------------------------------------------------------------------
// The stages' ring, turn by turn.
struct Turn {
  int st = 0;
  uint32_t phase = 0;
  MOE_DEVICE void next(int stages) {
    if (++st == stages) st = 0, phase ^= 1u;
  }
};

template <int R, int W, bool kFp16>
MOE_DEVICE void issue_shrink(const AdapterArgs& p, const Smem<R, W, kFp16>& s, const uint8_t* w, int rs, int n, uint32_t tmem) {
  using C = Cfg<R, W, kFp16>;
  const uint32_t wbytes = rs * 16 * 128, idesc = kFp16 ? idesc_f16_f32(s.tile_rows, 16 * rs) : idesc_bf16_f32(s.tile_rows, 16 * rs);
  const uint64_t pol = l2_policy_evict_last();
  const int xbytes = s.tile_rows * 128, stage = C::stage_bytes(s.tile_rows), stages = C::stages(s.tile_rows);
  const auto load = [&](int i, int st) {
    mbar_arrive_expect_tx(&s.full[st], wbytes);
    bulk_load(s.ring + st * stage + xbytes, w + static_cast<int64_t>(i) * C::kWBytes, wbytes, &s.full[st], pol);
  };
  fence_proxy_async_smem();  // (the ring was the tile search's memory)
  for (int i = 0; i < n && i < stages; ++i) load(i, i);
  Turn t, before;
  for (int i = 0; i < n; ++i, t.next(stages)) {
    if (!mbar_wait(&s.full[t.st], t.phase, s.abort_flag, p.err)) return;
    fence_proxy_async_smem();  // (x was written by the generic proxy)
    tc_fence_after();
    const uint32_t at = smem_u32(s.ring + t.st * stage);
    const uint64_t xd = operand_desc<128>(at), wd = operand_desc<128>(at + xbytes);
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_f16_ss(tmem + i % C::kAccs * R, xd + 2 * k, wd + 2 * k, idesc, i >= C::kAccs || k > 0);
    mma_commit(&s.empty[t.st]);
    if (i == 0) continue;
    // the stage of the step before is about to be free: its next A tile (x is asked for by the other warps)
    if (i - 1 + stages < n) {
      if (!mbar_wait(&s.empty[before.st], before.phase, s.abort_flag, p.err)) return;
      load(i - 1 + stages, before.st);
    }
    before.next(stages);
  }
  mma_commit(s.d_full);
}

template <int R, int W, bool kFp16>
MOE_DEVICE void load_b(const AdapterArgs& p, const Smem<R, W, kFp16>& s, const uint8_t* w, int j) {
  using C = Cfg<R, W, kFp16>;
  const int at = j % C::kBSlots;
  mbar_arrive_expect_tx(&s.b_full[at], C::kBTile);
  bulk_load(s.ring + C::b_at(at), w + static_cast<int64_t>(j) * C::kBTile, C::kBTile, &s.b_full[at],
            l2_policy_evict_last());
}

template <int R, int W, bool kFp16>
MOE_DEVICE void issue_expand(const AdapterArgs& p, const Smem<R, W, kFp16>& s, const uint8_t* w, int rs, int n, uint32_t tmem) {
  using C = Cfg<R, W, kFp16>;
  const uint32_t idesc = kFp16 ? idesc_f16_f32(s.tile_rows, kSlice) : idesc_bf16_f32(s.tile_rows, kSlice);
  const uint32_t u0 = smem_u32(s.u), b0 = smem_u32(s.ring);
  const int terms = u_terms<kFp16>(p);
  for (int j = C::kBEarly; j < n && j < C::kBSlots; ++j) load_b<R, W, kFp16>(p, s, w, j);  // (the partial sums' place is free now)
  for (int j = 0; j < n; ++j) {
    const int at = j % C::kBSlots, buf = j & 1;
    if (!mbar_wait(&s.b_full[at], (j / C::kBSlots) & 1, s.abort_flag, p.err)) return;
    if (!mbar_wait(&s.o_empty[buf], ((j >> 1) & 1) ^ 1, s.abort_flag, p.err)) return;
    tc_fence_after();
    for (int t = terms - 1; t >= 0; --t)  // (the small terms first: less of them is cut)
      for (int k = 0; k < rs; ++k) {  // 16 ranks: 32 bytes of a row, four to a block of 64 ranks
        const uint32_t in = (k / 4) * kRows * 128 + (k % 4) * 32;
        mma_f16_ss(tmem + buf * kSlice, operand_desc<C::kRowBytes>(u0 + t * C::kTerm + in),
                   operand_desc<C::kRowBytes>(b0 + C::b_at(at) + in), idesc, t < terms - 1 || k > 0);
      }
    mma_commit(&s.b_empty[at]);
    mma_commit(&s.o_full[buf]);
    if (j >= 1 && j - 1 + C::kBSlots < n) {
      if (!mbar_wait(&s.b_empty[(j - 1) % C::kBSlots], ((j - 1) / C::kBSlots) & 1, s.abort_flag, p.err)) return;
      load_b<R, W, kFp16>(p, s, w, j - 1 + C::kBSlots);
    }
  }
}

// ---- the other warps ---------------------------------------------------------------------------------------
// Arrives on the mbarrier (one of its expected arrivals) once this thread's copies so far have landed.
MOE_DEVICE void cp_async_mbar_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// x's rows into the stages: eight lanes a row's 128 bytes, 32 / W rows a lane.  The copies announce themselves; a proxy
// fence here, before each announcement, waited for every copy in flight and made the stages take turns (0.8 us each),
// so the issuing lane has it.
template <int R, int W, bool kFp16>
MOE_DEVICE void gather_x(const AdapterArgs& p, const Smem<R, W, kFp16>& s, int k0, int n) {
  using C = Cfg<R, W, kFp16>;
  const int piece = threadIdx.x & 7;
  constexpr int kPer = kRows / (4 * W);
  const uint16_t* row[kPer];
  uint32_t dst[kPer];
  bool live[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = (threadIdx.x >> 3) + 4 * W * i, t = s.rows[r];
    live[i] = t >= 0;  // (rows past the tile's last keep what the stage holds: their results go nowhere)
    row[i] = p.x + max(t, 0) * p.ldx + 64 * static_cast<int64_t>(k0);
    dst[i] = swizzled<128>(r, piece);
  }
  const int stage = C::stage_bytes(s.tile_rows), stages = C::stages(s.tile_rows);
  Turn t;
  for (int i = 0; i < n; ++i, t.next(stages)) {
    const int st = t.st;
    if (!mbar_wait_warp(&s.empty[st], t.phase ^ 1u, s.abort_flag, p.err)) return;
    uint8_t* at = s.ring + st * stage;
    const int col = 64 * (k0 + i) + 8 * piece;
    if (p.x_vec) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (live[j]) cp_async_16_part(smem_u32(at + dst[j]), col < p.K ? row[j] + 64 * i + 8 * piece : p.x, col < p.K ? 16u : 0u);
      cp_async_mbar_arrive(&s.full[st]);
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (live[j]) *reinterpret_cast<uint4*>(at + dst[j]) = load_x(row[j] - 64 * static_cast<int64_t>(k0), col, p.K);
      mbar_arrive(&s.full[st]);
    }
  }
}

// This CTA's partial sums (of `accs` accumulators) from TMEM into shared memory (16-byte units swizzled by the row).  D's
// rows lie a quarter in each warp's 32 TMEM lanes: 32, or the first 16 of them where M is 64.
template <int R>
MOE_DEVICE uint32_t part_at(int row, int unit) {
  constexpr int kMask = R / 4 < 8 ? R / 4 - 1 : 7;
  return (row * (R / 4) + (unit ^ (row & kMask))) * 16;
}
template <int R, int W, bool kFp16>
MOE_DEVICE void write_part(const Smem<R, W, kFp16>& s, uint32_t tmem, int accs) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = s.tile_rows / 4, row = per * (warp & 3) + lane;
  for (int c = 16 * (warp >> 2); c < R; c += 4 * W) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    for (int a = 0; a < accs; ++a) {
      uint32_t d[16];
      __syncwarp();  // (the load is the whole warp's, and lanes without a row skipped the stores before it)
      tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + a * R + c, d);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(d[i]);
    }
    if (lane < per) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(s.ring + part_at<R>(row, c / 4 + i)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  }
}

// u of this CTA's share of the rows, into every CTA of the cluster.
template <int R, int W, bool kFp16>
MOE_DEVICE void share_u(const AdapterArgs& p, const Smem<R, W, kFp16>& s, float scale, int rank, int rows, int cta) {
  using C = Cfg<R, W, kFp16>;
  // (whole warps take part, 256 / R rows each; those past the tile's last repeat it)
  const int share = (rows + p.cut.ctas - 1) / p.cut.ctas, terms = u_terms<kFp16>(p);
  for (int i = threadIdx.x * 8; (i & ~255) < share * R; i += 32 * W * 8) {
    const int r = min(min(i / R, share - 1) + cta * share, rows - 1), c = i % R;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    // (rows of 256 bytes and more: half of eight lanes take their second unit first, so that they meet no bank twice)
    const int swap = R >= 64 ? threadIdx.x >> 2 & 1 : 0;
    const uint32_t p0 = smem_u32(s.ring + part_at<R>(r, c / 4 + swap)), p1 = smem_u32(s.ring + part_at<R>(r, c / 4 + 1 - swap));
    for (int k = 0; k < p.cut.ctas; k += 4) {  // four CTAs' sums in flight
      float4 a[4], b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = b[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k + e < p.cut.ctas) a[e] = ld_cluster_f32x4(cluster_addr_u32(p0, k + e)), b[e] = ld_cluster_f32x4(cluster_addr_u32(p1, k + e));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[0] += a[e].x, v[1] += a[e].y, v[2] += a[e].z, v[3] += a[e].w;
        v[4] += b[e].x, v[5] += b[e].y, v[6] += b[e].z, v[7] += b[e].w;
      }
    }
    if (swap) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = v[e];
        v[e] = v[e + 4], v[e + 4] = x;
      }
    }
    uint4 term[kAdapterTerms<kFp16>];
    const float mul = adapter_split<R, kFp16>(v, c, rank, scale, term);
    const uint32_t at = smem_u32(s.u) + (c / 64) * kRows * 128 + swizzled<C::kRowBytes>(r, c % 64 / 8);
    for (int k = 0; k < p.cut.ctas; ++k) {
      const uint32_t to = cluster_addr_u32(at, k);
#pragma unroll
      for (int e = 0; e < kAdapterTerms<kFp16>; ++e)
        if (e < terms) st_cluster_v4(to + e * C::kTerm, term[e].x, term[e].y, term[e].z, term[e].w);
      if (kFp16 && c == 0) st_cluster_f32(cluster_addr(&s.row_scale[r], k), mul);
    }
  }
}

// The expand's steps: warp w has the rows of lane quarter w % 4 (32, or 16 of a 64-row tile) and the w / 4-th 32 (8 warps:
// 64) of the step's features, in units of 16 rows and 32 features.  The base of a unit is asked for four units (32-bit
// rows: two) before it is used: with two of 16-bit rows, 32 KB an SM, the memory's latency held the writes at 4.5 TB/s.
// kWhole: rows are 16-byte aligned and N is a multiple of 128: no column is checked.
template <typename E, int R, int W, bool kFp16, bool kWhole>
MOE_DEVICE void write_out(const AdapterArgs& p, const Smem<R, W, kFp16>& s, int s0, int n, uint32_t tmem) {
  constexpr int kCols = 512 / W, kChunks = kCols / 32, kUnits = 2 * kChunks;  // of a warp in a step
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int quarter = warp & 3, part = warp >> 2, per = s.tile_rows / 4;
  const bool has_base = p.base != nullptr;
  const int first = s0 * kSlice + kCols * part + 8 * q;  // this lane's column of the first step
  const E* base[2][2];
  E* out[2][2];
  float mul[2][2];
  bool live[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = per * quarter + 16 * m + 8 * h + g, r = 16 * m < per ? s.rows[at] : -1;
      live[m][h] = r >= 0;
      base[m][h] = static_cast<const E*>(has_base ? p.base : p.out) + max(r, 0) * (has_base ? p.ld_base : p.ld_out) + first;
      out[m][h] = static_cast<E*>(p.out) + max(r, 0) * p.ld_out + first;
      mul[m][h] = kFp16 && r >= 0 ? s.row_scale[at] : 1.0f;
    }
  const bool some[2] = {s.rows[per * quarter] >= 0, per > 16 && s.rows[per * quarter + 16] >= 0};  // (gaps come last)
  constexpr int kAhead = sizeof(E) == 2 ? 4 : 2;  // units, whole steps' or half a step's
  constexpr int kTurn = kAhead > kUnits ? kAhead / kUnits : 1;  // steps after which the units' places repeat
  Raw8<E> b[kAhead][2];
  // unit u (m = u / kChunks, chunk u % kChunks) of step j + ahead
  const auto ask = [&](int j, int ahead, int u, Raw8<E> (&to)[2]) {
    const int m = u / kChunks, off = ahead * kSlice + 32 * (u % kChunks);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = kWhole || (p.out_vec && first + j * kSlice + off < p.N);
      if (has_base && live[m][h] && j + ahead < n && in)
        to[h].load(base[m][h] + off);
      else
        to[h].zero();
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ask(0, i / kUnits, i % kUnits, b[i]);
  for (int j0 = 0; j0 < n; j0 += kTurn) {
#pragma unroll
    for (int i = 0; i < kTurn; ++i) {
      const int j = j0 + i, buf = j & 1;
      if (j >= n) break;
      if (!mbar_wait_warp(&s.o_full[buf], (j >> 1) & 1, s.abort_flag, p.err)) return;
      tc_fence_after();
      const uint32_t at = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + buf * kSlice + kCols * part;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int m = u / kChunks, c = u % kChunks, place = (i * kUnits + u) % kAhead;
        if (some[m]) {
          uint32_t d[16];
          __syncwarp();  // (the load is the whole warp's, and lanes without a row skipped the stores before it)
          tmem_ld_16x256b_x4(at + (static_cast<uint32_t>(16 * m) << 16) + 32 * c, d);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!live[m][h]) continue;
            float v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[2 * e] = __uint_as_float(d[4 * e + 2 * h]), v[2 * e + 1] = __uint_as_float(d[4 * e + 2 * h + 1]);
            const int col = first + j * kSlice + 32 * c;
            if (kWhole || p.out_vec) {
              float f[8];
              b[place][h].to_f32(f);
              if (kFp16) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], mul[m][h], f[e]);
              } else {
                add8(v, f);
              }
              if (kWhole || col < p.N) store8(out[m][h] + 32 * c, v);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (col + e < p.N) {
                  const float f = has_base ? base[m][h][32 * c + e].f32() : 0.0f;
                  out[m][h][32 * c + e] = E::of(kFp16 ? fmaf(v[e], mul[m][h], f) : v[e] + f);
                }
            }
          }
        }
        ask(j, (u + kAhead) / kUnits, (u + kAhead) % kUnits, b[place]);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) base[m][h] += kSlice, out[m][h] += kSlice;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o_empty[buf]);
    }
  }
}
template <typename E, int R, int W, bool kFp16>
MOE_DEVICE void write_out(const AdapterArgs& p, const Smem<R, W, kFp16>& s, int s0, int n, uint32_t tmem) {
  if (p.out_vec && p.N % kSlice == 0)
    write_out<E, R, W, kFp16, true>(p, s, s0, n, tmem);
  else
    write_out<E, R, W, kFp16, false>(p, s, s0, n, tmem);
}

// out = base (or zero) for a row: the bits, a warp a row.
MOE_DEVICE void copy_row(const AdapterArgs& p, int64_t row, int lane) {
  const int64_t e = p.out_type == MOE_FP32 ? 4 : 2, bytes = p.N * e;
  const uint8_t* from = p.base ? static_cast<const uint8_t*>(p.base) + row * p.ld_base * e : nullptr;
  uint8_t* to = static_cast<uint8_t*>(p.out) + row * p.ld_out * e;
  if (p.out_vec) {
    constexpr int kAhead = 8;
    for (int64_t i = lane * 16; i < bytes; i += 512 * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        v[k] = from && i + 512 * k < bytes ? *reinterpret_cast<const uint4*>(from + i + 512 * k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i + 512 * k < bytes) *reinterpret_cast<uint4*>(to + i + 512 * k) = v[k];
    }
  } else {
    for (int64_t i = lane * 2; i < bytes; i += 64)
      *reinterpret_cast<uint16_t*>(to + i) = from ? *reinterpret_cast<const uint16_t*>(from + i) : static_cast<uint16_t>(0);
  }
}

// What the cluster does: a tile (its rows in s.rows), or, behind the last tile, its share of the rows without an adapter
// (rank 0, t.rows of them from p.order[t.start], or in s.rows).  Every thread of the CTA calls it.
// From the grouping's list:
template <int R, int W, bool kFp16>
MOE_DEVICE void read_tile(const AdapterArgs& p, Smem<R, W, kFp16>& s, AdapterTile& t) {
  const int idx = blockIdx.x / p.cut.ctas;
  t = p.tiles[idx];  // (the list has an entry for every cluster of the grid)
  const int n = p.n_tiles[0], rest = p.n_tiles[1];
  s.tile_rows = p.n_tiles[2] <= 64 ? 64 : kRows;
  if (idx < n) {
    if (threadIdx.x < kRows) s.rows[threadIdx.x] = threadIdx.x < t.rows ? p.order[t.start + threadIdx.x] : -1;
  } else {
    const int clusters = gridDim.x / p.cut.ctas - n, share = (p.T - rest + clusters - 1) / clusters;
    t.start = min(rest + (idx - n) * share, p.T);
    s.spare = min(share, p.T - t.start);
    t.rank = 0;
  }
  __syncthreads();
}

// From the ids, by every CTA for itself: counts of all slots (no adapter counts as slot n), their tiles' scan, the slot
// that holds the cluster's tile, and that slot's rows in order.  Beside 64 x 64 products, 300 rows: 9.8 us, with the
// grouping's launch 12.0; 2051 rows: 13.6 and 13.4; 4096: 17.7 and 18.6, but 19.9 and 19.8 with two slots.
template <int R, int W, bool kFp16>
MOE_DEVICE void count_tile(const AdapterArgs& p, Smem<R, W, kFp16>& s, AdapterTile& t) {
  constexpr int kCounters = 32 * W;
  int* counts = reinterpret_cast<int*>(s.ring);     // [n + 1]
  int* warp_sum = counts + kAdaptersMax + 8;        // [W]
  int* pick = warp_sum + W;                // slot, tile within the slot, all tiles
  const int idx = blockIdx.x / p.cut.ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, most = p.cut.rows;
  const bool counter = tid < kCounters;
  s.tile_rows = most <= 64 ? 64 : kRows;
  for (int i = tid; i <= p.n; i += Cfg<R, W, kFp16>::kThreads) counts[i] = 0;
  if (tid == 0) pick[0] = p.n, pick[1] = 0;
  if (tid < kRows) s.rows[tid] = -1;
  __syncthreads();
  // a warp has a stretch of the step, whose ids stay in its lanes' registers
  constexpr int kIds = kAdapterCount / kCounters;
  const int stretch = (p.T + kCounters - 1) / kCounters, i0 = warp * 32 * stretch;
  int key[kIds];
#pragma unroll
  for (int j = 0; j < kIds; ++j) {
    const int i = i0 + 32 * j + lane;
    key[j] = -2;
    if (counter && j < stretch && i < p.T) {
      key[j] = p.ids[i];
      if (key[j] < 0 || key[j] >= p.n) {
        if (key[j] != -1 && blockIdx.x == 0) set_error(p.err, MOE_DEVERR_EXPERT_RANGE);
        key[j] = p.n;
      }
    }
  }
  if (counter) {
#pragma unroll
    for (int j = 0; j < kIds; ++j) count_key(counts, key[j], lane);
  }
  __syncthreads();
  // a counter's share of consecutive slots: its tiles, and those before it
  const int share = (p.n + kCounters - 1) / kCounters, first = min(tid * share, p.n), last = min(first + share, p.n);
  int mine = 0, upto = 0;
  if (counter) {
    for (int k = first; k < last; ++k) mine += (counts[k] + most - 1) / most;
    upto = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) warp_sum[warp] = upto;
  }
  __syncthreads();
  if (counter) {
    for (int w = 0; w < warp; ++w) upto += warp_sum[w];
    int at = upto - mine;
    if (idx >= at && idx < upto)
      for (int k = first; k < last; ++k) {
        const int tiles = (counts[k] + most - 1) / most;
        if (idx < at + tiles) {
          pick[0] = k, pick[1] = idx - at;
          break;
        }
        at += tiles;
      }
    if (tid == kCounters - 1) pick[2] = upto;
  }
  __syncthreads();
  // the rows of `slot` whose number lies in [from, from + rows)
  const int slot = pick[0], all = counts[slot];
  int from, rows;
  if (slot < p.n) {
    const int per = adapter_tile_rows(all, most);
    from = pick[1] * per, rows = min(per, all - from);
    t.rank = static_cast<uint16_t>(p.slots.rank[slot]), t.scale = p.slots.scale[slot];
  } else {  // behind the last tile: a share of the rows without an adapter, 128 at most (there are clusters enough)
    const int clusters = gridDim.x / p.cut.ctas - pick[2], per = (all + clusters - 1) / clusters;
    from = min((idx - pick[2]) * per, all), rows = min(per, all - from);
    t.rank = 0, t.scale = 0.0f;
  }
  t.slot = slot, t.start = -1, t.rows = static_cast<uint16_t>(rows);
  s.spare = rows;
  int number = 0;
  if (counter) {
#pragma unroll
    for (int j = 0; j < kIds; ++j) number += __popc(__ballot_sync(0xffffffffu, key[j] == slot));
    if (lane == 0) warp_sum[warp] = number;
  }
  __syncthreads();
  if (counter) {
    number = -from;
    for (int w = 0; w < warp; ++w) number += warp_sum[w];
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
      const uint32_t b = __ballot_sync(0xffffffffu, key[j] == slot);
      const int at = number + __popc(b & ((1u << lane) - 1u));
      if (key[j] == slot && at >= 0 && at < rows) s.rows[at] = i0 + 32 * j + lane;
      number += __popc(b);
    }
  }
  __syncthreads();  // (the ring's memory is free again, too)
}

template <int R, int W, bool kFp16>
__global__ void __launch_bounds__(Cfg<R, W, kFp16>::kThreads, Cfg<R, W, kFp16>::kCtas) adapter_tc_kernel(const AdapterArgs p) {
  using C = Cfg<R, W, kFp16>;
  extern __shared__ uint8_t smem_raw[];
  Smem<R, W, kFp16> s(smem_raw);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStagesMax; ++i) mbar_init(&s.full[i], 32 * W + 1), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < C::kBSlots; ++i) mbar_init(&s.b_full[i], 1), mbar_init(&s.b_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s.o_full[i], 1), mbar_init(&s.o_empty[i], W);
    mbar_init(s.d_full, 1);
    *s.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == W) {
    tmem_alloc(s.tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s.tmem_slot;
  pdl_trigger();  // (with its TMEM in hand: a dependent that came first would hold it while it waits for this grid)
  pdl_wait();
  const int cta = cluster_rank();
  AdapterTile t;
  if (p.tiles)
    read_tile(p, s, t);
  else
    count_tile(p, s, t);
  const int rank = t.rank, rs = (rank + 15) / 16;  // (the same for the whole cluster)
  if (rank == 0) {  // rows without an adapter, or of an empty slot: a warp a row, the cluster's warps in turn
    if (p.base != p.out) {
      const bool listed = t.start >= 0;
      const int rows = listed && blockIdx.x / p.cut.ctas < p.n_tiles[0] ? t.rows : s.spare;
      const int step = (W + 1) * p.cut.ctas;
      for (int i = warp * p.cut.ctas + cta; i < rows; i += step)
        copy_row(p, listed ? p.order[t.start + i] : s.rows[i], threadIdx.x & 31);
    }
  } else {
    const int nk = (p.K + 63) / 64, per_k = (nk + p.cut.ctas - 1) / p.cut.ctas, k0 = min(cta * per_k, nk), kn = min(per_k, nk - k0);
    const int ns = (p.N + kSlice - 1) / kSlice, per_n = (ns + p.cut.ctas - 1) / p.cut.ctas;
    const int s0 = min(cta * per_n, ns), sn = min(per_n, ns - s0);
    const uint8_t* wa = reinterpret_cast<const uint8_t*>(p.a_tc + t.slot * p.a_tc_slot) +
                        static_cast<int64_t>(k0) * C::kWBytes;
    const uint8_t* wb = reinterpret_cast<const uint8_t*>(p.b_tc + t.slot * p.b_tc_slot) +
                        static_cast<int64_t>(s0) * C::kBTile;
    if (warp == W) {
      // Few rows: the weights are most of what the tile reads, and come from memory: all of them are asked for now.
      // (With many rows an adapter's weights are in L2 already, and the requests cost 2 us of 15.)
      if (t.rows <= 32) {
        for (int j = threadIdx.x & 31; j < kn; j += 32) prefetch_l2(wa + static_cast<int64_t>(j) * C::kWBytes, rs * 16 * 128);
        for (int j = threadIdx.x & 31; j < sn; j += 32) prefetch_l2(wb + static_cast<int64_t>(j) * C::kBTile, C::kBTile);
      }
      __syncwarp();
      if (elect_one() && kn > 0) {
        issue_shrink<R, W, kFp16>(p, s, wa, rs, kn, tmem);
        // the ring is free once the shrink's MMAs are done: B's first tiles, behind the partial sums' place
        if (mbar_wait(s.d_full, 0, s.abort_flag, p.err))
          for (int j = 0; j < sn && j < C::kBEarly; ++j) load_b<R, W, kFp16>(p, s, wb, j);
      }
      __syncwarp();
      if (kn == 0 && elect_one())
        for (int j = 0; j < sn && j < C::kBEarly; ++j) load_b<R, W, kFp16>(p, s, wb, j);
      __syncwarp();
    } else {
      gather_x<R, W, kFp16>(p, s, k0, kn);
      const bool done = kn > 0 && mbar_wait_warp(s.d_full, 0, s.abort_flag, p.err);
      tc_fence_after();
      write_part<R, W, kFp16>(s, tmem, done ? min(kn, C::kAccs) : 0);
      tc_fence_before();
    }
    cluster_barrier();
    if (warp < W) share_u<R, W, kFp16>(p, s, t.scale, rank, t.rows, cta);
    fence_proxy_async_all();
    cluster_barrier();  // u is whole, and no CTA's partial sums are read any more
    tc_fence_after();
    fence_proxy_async_all();
    if (warp == W) {
      if (elect_one()) issue_expand<R, W, kFp16>(p, s, wb, rs, sn, tmem);
      __syncwarp();
    } else if (p.out_type == MOE_BF16) {
      write_out<Bf16, R, W, kFp16>(p, s, s0, sn, tmem);
    } else if (p.out_type == MOE_FP16) {
      write_out<Fp16, R, W, kFp16>(p, s, s0, sn, tmem);
    } else {
      write_out<Fp32, R, W, kFp16>(p, s, s0, sn, tmem);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  abort_quiesce(s.abort_flag);
  if (warp == W) tmem_dealloc(tmem, C::kTmemCols);
}

// ---- packing -------------------------------------------------------------------------------------------
// A: 64 columns at a time, [R rows][128 bytes] swizzled.  B: 128 features at a time, blocks of 64 ranks
// [128 rows][kRowBytes] swizzled; row 8 i + 2 q + b of each 32 is feature 8 q + 2 i + b.
template <int R>
__global__ void adapter_tc_pack_kernel(const uint16_t* a, const uint16_t* b, uint16_t* pa, uint16_t* pb, int r, int K, int N,
                                       int64_t na, int64_t nb) {
  using C = Cfg<R, 16, true>;
  constexpr int W = C::kRowBytes / 2;  // elements of a row
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < na + nb;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    if (i < na) {
      const int64_t chunk = i / (64 * R);
      const int row = i / 64 % R, e = i % 64;
      const int64_t col = 64 * chunk + e;
      pa[chunk * (64 * R) + swizzled<128>(row, e / 8) / 2 + e % 8] =
          row < r && col < K ? a[row * static_cast<int64_t>(K) + col] : 0;
    } else {
      const int64_t o = i - na, tile = o / (kSlice * R);
      const int in = o % (kSlice * R), block = in / (kSlice * W), row = in / W % kSlice, e = in % W;
      const int x = row % 32, rank = 64 * block + e;
      const int64_t f = kSlice * tile + 32 * (row / 32) + 8 * (x / 2 % 4) + 2 * (x / 8) + x % 2;
      pb[tile * (kSlice * R) + block * (kSlice * W) + swizzled<C::kRowBytes>(row, e / 8) / 2 + e % 8] =
          rank < r && f < N ? b[f * r + rank] : 0;
    }
  }
}

template <int R>
cudaError_t pack(const uint16_t* a, const uint16_t* b, uint16_t* pa, uint16_t* pb, int r, int K, int N, cudaStream_t st) {
  const int64_t na = adapter_tc_a_elems(K, R), nb = adapter_tc_b_elems(N, R), blocks = (na + nb + 255) / 256;
  adapter_tc_pack_kernel<R><<<static_cast<int>(blocks < 4096 ? blocks : 4096), 256, 0, st>>>(a, b, pa, pb, r, K, N, na, nb);
  return cudaGetLastError();
}

template <int R, int W, bool kFp16>
cudaError_t launch_warps(const AdapterArgs& p, cudaStream_t st) {
  auto kern = adapter_tc_kernel<R, W, kFp16>;
  using C = Cfg<R, W, kFp16>;
  cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::kBytes);
  if (e != cudaSuccess) return e;
  const int clusters = adapter_clusters(p.T, p.n, p.cut, p.base != p.out);
  return launch_pdl_clusters(kern, dim3(clusters * p.cut.ctas), dim3(C::kThreads), p.cut.ctas, C::kBytes, st, p);
}

template <int R, bool kFp16>
cudaError_t launch(const AdapterArgs& p, cudaStream_t st) {
  if constexpr (R <= 64) {
    if (p.cut.small) return launch_warps<R, 8, kFp16>(p, st);
  }
  return launch_warps<R, 16, kFp16>(p, st);
}

}  // namespace

cudaError_t launch_adapter_tc_pack(const uint16_t* a, const uint16_t* b, uint16_t* pa, uint16_t* pb, int r, int K, int N,
                                   int rpad, cudaStream_t st) {
  switch (rpad) {
    case 16: return pack<16>(a, b, pa, pb, r, K, N, st);
    case 32: return pack<32>(a, b, pa, pb, r, K, N, st);
    case 64: return pack<64>(a, b, pa, pb, r, K, N, st);
    default: return pack<128>(a, b, pa, pb, r, K, N, st);
  }
}

// Up to 3500 rows two CTAs of 8 warps run on an SM, whose waits fill each other, above one of 16 with a deep ring.  Both, us,
// two CTAs first, in 8 slots (in 64), a tenth of the rows without an adapter:
//     rows               1500                     3500                     5000                     8000
//     rank 64, 4096x4096 25.2 34.7 (33.9 37.9)    36.2 36.0 (48.4 39.6)    54.1 42.5 (57.1 47.2)    59.6 47.1 (91.6 60.1)
//     rank 16, 2048x4096 19.0 27.2 (22.5 27.8)    25.4 34.1 (34.4 30.2)    36.5 37.6 (37.4 38.0)    42.3 40.3 (58.4 48.4)
//     rank 16, 1024x1024 14.0 19.7 (14.6 16.1)    15.5 21.6 (17.6 17.8)    18.8 19.0 (18.9 20.3)    20.5 20.1 (26.2 23.1)
// CTAs that share a tile: a power of two that should leave all tiles running at once.  How many there will be is unknown here:
// a slot that has rows has a tile at least, and loses part of one.  (8195 rows in 32 slots, one of 16 warps: 52 us with 2 CTAs
// a tile and 60 with 1 where 64 tiles come out, 67 and 60 where 80 do.)
AdapterCut adapter_cut(int T, int n, int rpad, int num_sms) {
  const int used = n < T ? n : T;
  AdapterCut c;
  c.small = rpad <= 64 && T <= 3500;
  c.slots = c.small ? 2 * num_sms : num_sms;
  const int about = c.small ? T / 64 + used / 2 + 1 : T / kRows + used / 4 + 1, tiles = about > used ? about : used;
  c.ctas = 8;
  while (c.ctas > 1 && tiles * c.ctas > c.slots) c.ctas /= 2;
  // (steps with a grouping launch: it chooses the rows)
  c.rows = static_cast<int64_t>(T / 64 + used / 2 + 1) * c.ctas <= c.slots ? 64 : kRows;
  return c;
}

// Clusters of the grid: for all tiles that there may be, of the rows that the grouping may choose to fill whole waves (64 at
// least), and a few more where there may be rows to be copied.  (A cluster with nothing to do costs its CTAs' start.)
int adapter_clusters(int T, int n, const AdapterCut& cut, bool copies) {
  const int64_t used = n < T ? n : T, most = (T + cut.rows - 1) / cut.rows + used;
  const int64_t waves = (most * cut.ctas + cut.slots - 1) / cut.slots, whole = waves * cut.slots / cut.ctas;
  const int64_t fine = (T + 63) / 64 + used, tiles = most > whole ? most : whole < fine ? whole : fine;
  return static_cast<int>((most > tiles ? most : tiles) + (copies ? cut.slots / (8 * cut.ctas) + 1 : 0));
}

cudaError_t launch_adapters_tc(const AdapterArgs& p, int rpad, bool fp16, cudaStream_t st) {
  switch (rpad) {
    case 16: return fp16 ? launch<16, true>(p, st) : launch<16, false>(p, st);
    case 32: return fp16 ? launch<32, true>(p, st) : launch<32, false>(p, st);
    case 64: return fp16 ? launch<64, true>(p, st) : launch<64, false>(p, st);
    default: return fp16 ? launch<128, true>(p, st) : launch<128, false>(p, st);
  }
}

}  // namespace moe
