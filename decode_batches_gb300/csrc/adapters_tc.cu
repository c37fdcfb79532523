// Low-rank adapters of larger steps on the tensor cores (adapters.cu has the formulas and the small steps' kernel).
//
// A tile is up to 128 rows of one adapter, a cluster of C CTAs computes it:
//   shrink  D[128][R] = x A^T over this CTA's range of K: tcgen05 MMAs of 128 x R x 16, rows of x gathered with cp.async
//           into the 128-byte-swizzled operand, A in tiles packed that way (bulk copies), a ring of 64-column stages;
//   u       the CTAs' partial sums meet in distributed shared memory: each CTA adds up 128 / C rows, scales and splits
//           them into two 16-bit terms (adapter_split) and writes those into every CTA's MMA operand;
//   expand  128 features at a time, over this CTA's range of N: D[128][128] = (hi + lo) B^T, two MMAs a 16 ranks, D double
//           buffered in TMEM; eight warps add the base and write.
// Bound by memory: x, base and out pass once; the weights are read once a tile, from L2.  What the warp-level kernel's
// fragments cost (24 M instructions for 8195 rows of 4096 x 4096, rank 64: 75 us) falls away: operands go from shared
// memory to the tensor core without registers.
//
// The rows of a B tile are permuted within 32 features such that the 16x256b TMEM load hands a lane eight neighbouring
// features of a row: base and out move as 16-byte vectors, 64 contiguous bytes a row, without a transposition.
#include "adapters.cuh"
#include "adapters_split.cuh"
#include "cluster.cuh"
#include "elems.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;             // rows of a tile (the MMA's M)
constexpr int kMathWarps = 8;          // gather, reduction, epilogue
constexpr int kThreads = 32 * (kMathWarps + 1);
constexpr int kSlice = 128;            // features of an expand step
constexpr int kStagesMax = 8;

// Shared memory: the ring, then u.  During the shrink its stages run on into u's place; after it the ring's start holds
// the partial sums, B's first tiles come behind them and the later ones, once the sums are read, also in their place.
template <int R>
struct Cfg {
  static constexpr int kWBytes = R * 128;
  static constexpr int kTerm = kRows * R * 2;        // u's hi or lo
  static constexpr int kPart = kRows * R * 4;        // partial sums
  static constexpr int kBTile = kSlice * R * 2;
  static constexpr int kRing = R <= 64 ? 72 * 1024 : 128 * 1024;  // (two CTAs an SM up to rank 64)
  static constexpr int kBEarly = (kRing - kPart) / kBTile < 4 ? (kRing - kPart) / kBTile : 4;
  static constexpr int kBSlots = kBEarly + kPart / kBTile;
  static constexpr int kRowBytes = (R < 64 ? R : 64) * 2;  // a row of u or of a B tile within a block of 64 ranks
  static constexpr int kTail = kRows * 8 + 320;
  static constexpr int kBytes = kRing + 2 * kTerm + kTail + 1024;
  static constexpr int kTmemCols = 256;              // two buffers of 128; the shrink's R are the first's
  static constexpr int b_at(int slot) { return slot < kBEarly ? kPart + slot * kBTile : (slot - kBEarly) * kBTile; }
  static_assert(kBEarly >= 2 && kBSlots <= 6, "");
  // Stages for tiles of `rows` rows (64 or 128).  With 64 the MMA's other 64 rows are whatever follows, so that the last
  // stage's 16 KB have to end within the memory: 6 stages of 16 KB instead of 4 of 24 at rank 64, the same bytes of x in
  // flight as with whole tiles and half as many again as with half-empty stages.
  static constexpr int stage_bytes(int rows) { return rows * 128 + kWBytes; }
  static constexpr int stages(int rows) {
    const int n = (kRing + 2 * kTerm - kRows * 128) / stage_bytes(rows) + 1, m = (kRing + 2 * kTerm) / stage_bytes(rows);
    return n < m ? (n < kStagesMax ? n : kStagesMax) : (m < kStagesMax ? m : kStagesMax);
  }
};

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

template <int R>
struct Smem {
  uint8_t* ring;
  uint8_t* u;
  int* rows;         // [128] row numbers, -1 past the last
  float* row_scale;  // [128] (fp16)
  uint64_t* full;    // [kStagesMax] x's 256 threads and A's copy
  uint64_t* empty;   // [kStagesMax]
  uint64_t* b_full;  // [kBSlots]
  uint64_t* b_empty;
  uint64_t* o_full;  // [2] D of an expand step
  uint64_t* o_empty;
  uint64_t* d_full;  // the shrink's D
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  MOE_DEVICE explicit Smem(uint8_t* raw) {
    uint8_t* p = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    ring = p, p += Cfg<R>::kRing;
    u = p, p += 2 * Cfg<R>::kTerm;
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

template <int R, bool kFp16>
MOE_DEVICE void issue_shrink(const AdapterArgs& p, const Smem<R>& s, const uint8_t* w, int rs, int n, uint32_t tmem) {
  using C = Cfg<R>;
  const uint32_t wbytes = rs * 16 * 128, idesc = kFp16 ? idesc_f16_f32(kRows, 16 * rs) : idesc_bf16_f32(kRows, 16 * rs);
  const uint64_t pol = l2_policy_evict_last();
  const int xbytes = p.cut.rows * 128, stage = C::stage_bytes(p.cut.rows), stages = C::stages(p.cut.rows);
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
    for (int k = 0; k < 4; ++k) mma_f16_ss(tmem, xd + 2 * k, wd + 2 * k, idesc, i > 0 || k > 0);
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

template <int R>
MOE_DEVICE void load_b(const AdapterArgs& p, const Smem<R>& s, const uint8_t* w, int j) {
  using C = Cfg<R>;
  const int at = j % C::kBSlots;
  mbar_arrive_expect_tx(&s.b_full[at], C::kBTile);
  bulk_load(s.ring + C::b_at(at), w + static_cast<int64_t>(j) * C::kBTile, C::kBTile, &s.b_full[at],
            l2_policy_evict_last());
}

template <int R, bool kFp16>
MOE_DEVICE void issue_expand(const AdapterArgs& p, const Smem<R>& s, const uint8_t* w, int rs, int n, uint32_t tmem) {
  using C = Cfg<R>;
  const uint32_t idesc = kFp16 ? idesc_f16_f32(kRows, kSlice) : idesc_bf16_f32(kRows, kSlice);
  const uint32_t u0 = smem_u32(s.u), b0 = smem_u32(s.ring);
  for (int j = C::kBEarly; j < n && j < C::kBSlots; ++j) load_b<R>(p, s, w, j);  // (the partial sums' place is free now)
  for (int j = 0; j < n; ++j) {
    const int at = j % C::kBSlots, buf = j & 1;
    if (!mbar_wait(&s.b_full[at], (j / C::kBSlots) & 1, s.abort_flag, p.err)) return;
    if (!mbar_wait(&s.o_empty[buf], ((j >> 1) & 1) ^ 1, s.abort_flag, p.err)) return;
    tc_fence_after();
    for (int t = 0; t < 2; ++t)
      for (int k = 0; k < rs; ++k) {  // 16 ranks: 32 bytes of a row, four to a block of 64 ranks
        const uint32_t in = (k / 4) * kRows * 128 + (k % 4) * 32;
        mma_f16_ss(tmem + buf * kSlice, operand_desc<C::kRowBytes>(u0 + t * C::kTerm + in),
                   operand_desc<C::kRowBytes>(b0 + C::b_at(at) + in), idesc, t > 0 || k > 0);
      }
    mma_commit(&s.b_empty[at]);
    mma_commit(&s.o_full[buf]);
    if (j >= 1 && j - 1 + C::kBSlots < n) {
      if (!mbar_wait(&s.b_empty[(j - 1) % C::kBSlots], ((j - 1) / C::kBSlots) & 1, s.abort_flag, p.err)) return;
      load_b<R>(p, s, w, j - 1 + C::kBSlots);
    }
  }
}

// Asks L2 for `bytes` from p (16-byte aligned, a multiple of 16).
MOE_DEVICE void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// ---- the other warps ---------------------------------------------------------------------------------------
// Arrives on the mbarrier (one of its expected arrivals) once this thread's copies so far have landed.
MOE_DEVICE void cp_async_mbar_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// x's rows into the stages: eight lanes a row's 128 bytes, four rows a lane.  The copies announce themselves; a proxy
// fence here, before each announcement, waited for every copy in flight and made the stages take turns (0.8 us each),
// so the issuing lane has it.
template <int R>
MOE_DEVICE void gather_x(const AdapterArgs& p, const Smem<R>& s, int k0, int n) {
  using C = Cfg<R>;
  const int piece = threadIdx.x & 7;
  const uint16_t* row[4];
  uint32_t dst[4];
  bool live[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (threadIdx.x >> 3) + 32 * i, t = s.rows[r];
    live[i] = t >= 0;  // (rows past the tile's last keep what the stage holds: their results go nowhere)
    row[i] = p.x + max(t, 0) * p.ldx + 64 * static_cast<int64_t>(k0);
    dst[i] = swizzled<128>(r, piece);
  }
  const int stage = C::stage_bytes(p.cut.rows), stages = C::stages(p.cut.rows);
  Turn t;
  for (int i = 0; i < n; ++i, t.next(stages)) {
    const int st = t.st;
    if (!mbar_wait_warp(&s.empty[st], t.phase ^ 1u, s.abort_flag, p.err)) return;
    uint8_t* at = s.ring + st * stage;
    const int col = 64 * (k0 + i) + 8 * piece;
    if (p.x_vec) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (live[j]) cp_async_16_part(smem_u32(at + dst[j]), col < p.K ? row[j] + 64 * i + 8 * piece : p.x, col < p.K ? 16u : 0u);
      cp_async_mbar_arrive(&s.full[st]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (live[j]) *reinterpret_cast<uint4*>(at + dst[j]) = load_x(row[j] - 64 * static_cast<int64_t>(k0), col, p.K);
      mbar_arrive(&s.full[st]);
    }
  }
}

// This CTA's partial sums from TMEM into shared memory (16-byte units swizzled by the row).
template <int R>
MOE_DEVICE uint32_t part_at(int row, int unit) {
  constexpr int kMask = R / 4 < 8 ? R / 4 - 1 : 7;
  return (row * (R / 4) + (unit ^ (row & kMask))) * 16;
}
template <int R>
MOE_DEVICE void write_part(const Smem<R>& s, uint32_t tmem, bool any) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = 32 * (warp & 3) + lane;
  for (int c = 16 * (warp >> 2); c < R; c += 32) {
    uint32_t v[16];
    if (any) {
      tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c, v);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(s.ring + part_at<R>(row, c / 4 + i)) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

// u of this CTA's share of the rows, into every CTA of the cluster.
template <int R, bool kFp16>
MOE_DEVICE void share_u(const AdapterArgs& p, const Smem<R>& s, float scale, int rank, int rows, int cta) {
  using C = Cfg<R>;
  // (whole warps take part, 256 / R rows each; those past the tile's last repeat it)
  const int share = (rows + p.cut.ctas - 1) / p.cut.ctas;
  for (int i = threadIdx.x * 8; (i & ~255) < share * R; i += 32 * kMathWarps * 8) {
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
    uint4 hi, lo;
    const float mul = adapter_split<R, kFp16>(v, c, rank, scale, hi, lo);
    const uint32_t at = smem_u32(s.u) + (c / 64) * kRows * 128 + swizzled<C::kRowBytes>(r, c % 64 / 8);
    for (int k = 0; k < p.cut.ctas; ++k) {
      const uint32_t to = cluster_addr_u32(at, k);
      st_cluster_v4(to, hi.x, hi.y, hi.z, hi.w);
      st_cluster_v4(to + C::kTerm, lo.x, lo.y, lo.z, lo.w);
      if (kFp16 && c == 0) st_cluster_f32(cluster_addr(&s.row_scale[r], k), mul);
    }
  }
}

// The expand's steps: warp w has the rows of lane quarter w % 4 and half w / 4 of the step's features.  A step is four
// units of 16 rows and 32 features.  The base of a unit is asked for kAhead units before it is used: with two units of
// 16-bit rows in flight a warp, 32 KB an SM, the memory's latency held the writes at 4.5 TB/s.
// kWhole: rows are 16-byte aligned and N is a multiple of 128: no column is checked.
template <typename E, int R, bool kFp16, bool kWhole>
MOE_DEVICE void write_out(const AdapterArgs& p, const Smem<R>& s, int s0, int n, int rank, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int quarter = warp & 3, half = warp >> 2;
  const bool has_base = p.base != nullptr;
  const int first = s0 * kSlice + 64 * half + 8 * q;  // this lane's column of a step's first units
  const E* base[2][2];
  E* out[2][2];
  float mul[2][2];
  bool live[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = 32 * quarter + 16 * m + 8 * h + g, r = s.rows[at];
      live[m][h] = r >= 0;
      base[m][h] = static_cast<const E*>(has_base ? p.base : p.out) + max(r, 0) * (has_base ? p.ld_base : p.ld_out) + first;
      out[m][h] = static_cast<E*>(p.out) + max(r, 0) * p.ld_out + first;
      mul[m][h] = kFp16 && rank > 0 ? s.row_scale[at] : 1.0f;
    }
  const bool some[2] = {s.rows[32 * quarter] >= 0, s.rows[32 * quarter + 16] >= 0};  // (rows come first, gaps last)
  constexpr int kAhead = sizeof(E) == 2 ? 4 : 2;
  Raw8<E> b[kAhead][2];
  // unit `unit` of the step `next` steps on
  const auto ask = [&](int j, int next, int unit, Raw8<E> (&to)[2]) {
    const int m = unit >> 1, off = next * kSlice + 32 * (unit & 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = kWhole || (p.out_vec && first + j * kSlice + off < p.N);
      if (has_base && live[m][h] && j + next < n && in)
        to[h].load(base[m][h] + off);
      else
        to[h].zero();
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ask(0, 0, i, b[i]);
  for (int j = 0; j < n; ++j) {
    const int buf = j & 1;
    if (rank > 0) {
      if (!mbar_wait_warp(&s.o_full[buf], (j >> 1) & 1, s.abort_flag, p.err)) return;
      tc_fence_after();
    }
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + buf * kSlice + 64 * half;
#pragma unroll
    for (int unit = 0; unit < 4; ++unit) {
      const int m = unit >> 1, c = unit & 1;
      if (some[m]) {
        uint32_t d[16];
        if (rank > 0) {
          tmem_ld_16x256b_x4(at + (static_cast<uint32_t>(16 * m) << 16) + 32 * c, d);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) d[i] = 0u;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!live[m][h]) continue;
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[2 * i] = __uint_as_float(d[4 * i + 2 * h]), v[2 * i + 1] = __uint_as_float(d[4 * i + 2 * h + 1]);
          if (kWhole || p.out_vec) {
            float f[8];
            b[unit % kAhead][h].to_f32(f);
            if (kFp16) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], mul[m][h], f[i]);
            } else {
              add8(v, f);
            }
            if (kWhole || first + j * kSlice + 32 * c < p.N) store8(out[m][h] + 32 * c, v);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (first + j * kSlice + 32 * c + i < p.N) {
                const float f = has_base ? base[m][h][32 * c + i].f32() : 0.0f;
                out[m][h][32 * c + i] = E::of(kFp16 ? fmaf(v[i], mul[m][h], f) : v[i] + f);
              }
          }
        }
      }
      ask(j, unit + kAhead < 4 ? 0 : 1, (unit + kAhead) % 4, b[unit % kAhead]);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) base[m][h] += kSlice, out[m][h] += kSlice;
    if (rank > 0) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o_empty[buf]);
    }
  }
}
template <typename E, int R, bool kFp16>
MOE_DEVICE void write_out(const AdapterArgs& p, const Smem<R>& s, int s0, int n, int rank, uint32_t tmem) {
  if (p.out_vec && p.N % kSlice == 0)
    write_out<E, R, kFp16, true>(p, s, s0, n, rank, tmem);
  else
    write_out<E, R, kFp16, false>(p, s, s0, n, rank, tmem);
}

// The cluster's tile and its rows (to s.rows) from the grouping's list.  Every thread of the CTA calls it.
template <int R>
MOE_DEVICE bool read_tile(const AdapterArgs& p, const Smem<R>& s, AdapterTile& t) {
  const int idx = blockIdx.x / p.cut.ctas, n = *p.n_tiles;
  t = p.tiles[idx];  // (the list has an entry for every cluster of the grid)
  if (idx >= n) return false;
  if (threadIdx.x < kRows) s.rows[threadIdx.x] = threadIdx.x < t.rows ? p.order[t.start + threadIdx.x] : -1;
  __syncthreads();
  return true;
}

// The same from the ids, by every CTA for itself: counts of all slots (no adapter counts as slot n), their tiles' scan,
// the slot that holds the cluster's tile, and that slot's rows in order.  Beside 64 x 64 products, 300 rows: 9.8 us, with
// the grouping's launch 12.0; 2051 rows: 13.6 and 13.4; 4096: 17.7 and 18.6, but 19.9 and 19.8 with two slots.
template <int R>
MOE_DEVICE bool count_tile(const AdapterArgs& p, const Smem<R>& s, AdapterTile& t) {
  constexpr int kCounters = 32 * kMathWarps;
  int* counts = reinterpret_cast<int*>(s.ring);     // [n + 1]
  int* warp_sum = counts + kAdaptersMax + 8;        // [8]
  int* pick = warp_sum + kMathWarps;                // slot, rows of the slot, tile within the slot
  const int idx = blockIdx.x / p.cut.ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool counter = tid < kCounters;
  for (int i = tid; i <= p.n; i += kThreads) counts[i] = 0;
  if (tid == 0) pick[0] = -1;
  if (tid < kRows) s.rows[tid] = -1;
  __syncthreads();
  // a warp has a stretch of the step, whose ids stay in its lanes' registers
  constexpr int kIds = kAdapterCount / kCounters;
  const int stretch = (p.T + kCounters - 1) / kCounters, i0 = warp * 32 * stretch;
  int key[kIds];
#pragma unroll
  for (int j = 0; j < kIds; ++j) {
    const int i = i0 + 32 * j + lane;
    key[j] = counter && j < stretch && i < p.T ? p.ids[i] : -2;
  }
  if (counter) {
    bool bad_id = false;
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
      if (j >= stretch) break;
      if (key[j] != -2 || i0 + 32 * j + lane < p.T) {
        if (key[j] < 0 || key[j] >= p.n) bad_id |= key[j] != -1, key[j] = p.n;
      }
      count_key(counts, key[j], lane);
    }
    if (bad_id && blockIdx.x == 0) set_error(p.err, MOE_DEVERR_EXPERT_RANGE);
  }
  __syncthreads();
  // a counter's share of consecutive slots: its tiles, and those before it
  const int share = (p.n + 1 + kCounters - 1) / kCounters, first = tid * share, last = min(first + share, p.n + 1);
  int mine = 0, upto = 0;
  if (counter) {
    for (int k = first; k < last; ++k) mine += (counts[k] + p.cut.rows - 1) / p.cut.rows;
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
        const int tiles = (counts[k] + p.cut.rows - 1) / p.cut.rows;
        if (idx < at + tiles) {
          pick[0] = k, pick[1] = counts[k], pick[2] = idx - at;
          break;
        }
        at += tiles;
      }
  }
  __syncthreads();
  const int slot = pick[0], all = pick[1];
  if (slot < 0) return false;
  const int per = adapter_tile_rows(all, p.cut.rows), from = pick[2] * per;
  t.slot = slot < p.n ? slot : -1, t.start = 0, t.rows = static_cast<uint16_t>(min(per, all - from));
  t.rank = slot < p.n ? static_cast<uint16_t>(p.slots.rank[slot]) : 0;
  t.scale = slot < p.n ? p.slots.scale[slot] : 0.0f;
  // each warp numbers the slot's rows of its stretch
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
      if (key[j] == slot && at >= 0 && at < t.rows) s.rows[at] = i0 + 32 * j + lane;
      number += __popc(b);
    }
  }
  __syncthreads();  // (the ring's memory is free again, too)
  return true;
}

template <int R, bool kFp16>
__global__ void __launch_bounds__(kThreads, R <= 64 ? 2 : 1) adapter_tc_kernel(const AdapterArgs p) {
  using C = Cfg<R>;
  extern __shared__ uint8_t smem_raw[];
  const Smem<R> s(smem_raw);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStagesMax; ++i) mbar_init(&s.full[i], 32 * kMathWarps + 1), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < C::kBSlots; ++i) mbar_init(&s.b_full[i], 1), mbar_init(&s.b_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s.o_full[i], 1), mbar_init(&s.o_empty[i], kMathWarps);
    mbar_init(s.d_full, 1);
    *s.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMathWarps) {
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
  const bool found = p.tiles ? read_tile(p, s, t) : count_tile(p, s, t);
  const int rank = t.rank, rs = (rank + 15) / 16;
  if (found && !(rank == 0 && p.base == p.out)) {  // (the same for the whole cluster)
    const int nk = (p.K + 63) / 64, per_k = (nk + p.cut.ctas - 1) / p.cut.ctas, k0 = min(cta * per_k, nk), kn = min(per_k, nk - k0);
    const int ns = (p.N + kSlice - 1) / kSlice, per_n = (ns + p.cut.ctas - 1) / p.cut.ctas;
    const int s0 = min(cta * per_n, ns), sn = min(per_n, ns - s0);
    const uint8_t* wa = reinterpret_cast<const uint8_t*>(p.a_tc + (rank > 0 ? t.slot * p.a_tc_slot : 0)) +
                        static_cast<int64_t>(k0) * C::kWBytes;
    const uint8_t* wb = reinterpret_cast<const uint8_t*>(p.b_tc + (rank > 0 ? t.slot * p.b_tc_slot : 0)) +
                        static_cast<int64_t>(s0) * C::kBTile;
    if (rank > 0) {
      if (warp == kMathWarps) {
        // Few rows: the weights are most of what the tile reads, and come from memory: all of them are asked for now.
        // (With many rows an adapter's weights are in L2 already, and the requests cost 2 us of 15.)
        if (t.rows <= 32) {
          for (int j = threadIdx.x & 31; j < kn; j += 32) prefetch_l2(wa + static_cast<int64_t>(j) * C::kWBytes, rs * 16 * 128);
          for (int j = threadIdx.x & 31; j < sn; j += 32) prefetch_l2(wb + static_cast<int64_t>(j) * C::kBTile, C::kBTile);
        }
        __syncwarp();
        if (elect_one() && kn > 0) {
          issue_shrink<R, kFp16>(p, s, wa, rs, kn, tmem);
          // the ring is free once the shrink's MMAs are done: B's first tiles, behind the partial sums' place
          if (mbar_wait(s.d_full, 0, s.abort_flag, p.err))
            for (int j = 0; j < sn && j < C::kBEarly; ++j) load_b<R>(p, s, wb, j);
        }
        __syncwarp();
        if (kn == 0 && elect_one())
          for (int j = 0; j < sn && j < C::kBEarly; ++j) load_b<R>(p, s, wb, j);
        __syncwarp();
      } else {
        gather_x<R>(p, s, k0, kn);
        const bool done = kn > 0 && mbar_wait_warp(s.d_full, 0, s.abort_flag, p.err);
        tc_fence_after();
        write_part<R>(s, tmem, done);
        tc_fence_before();
      }
      cluster_barrier();
      if (warp < kMathWarps) share_u<R, kFp16>(p, s, t.scale, rank, t.rows, cta);
      fence_proxy_async_all();
      cluster_barrier();  // u is whole, and no CTA's partial sums are read any more
      tc_fence_after();
      fence_proxy_async_all();
    }
    if (warp == kMathWarps) {
      if (rank > 0 && elect_one()) issue_expand<R, kFp16>(p, s, wb, rs, sn, tmem);
      __syncwarp();
    } else if (p.out_type == MOE_BF16) {
      write_out<Bf16, R, kFp16>(p, s, s0, sn, rank, tmem);
    } else if (p.out_type == MOE_FP16) {
      write_out<Fp16, R, kFp16>(p, s, s0, sn, rank, tmem);
    } else {
      write_out<Fp32, R, kFp16>(p, s, s0, sn, rank, tmem);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  abort_quiesce(s.abort_flag);
  if (warp == kMathWarps) tmem_dealloc(tmem, C::kTmemCols);
}

// ---- packing -------------------------------------------------------------------------------------------
// A: 64 columns at a time, [R rows][128 bytes] swizzled.  B: 128 features at a time, blocks of 64 ranks
// [128 rows][kRowBytes] swizzled; row 8 i + 2 q + b of each 32 is feature 8 q + 2 i + b.
template <int R>
__global__ void adapter_tc_pack_kernel(const uint16_t* a, const uint16_t* b, uint16_t* pa, uint16_t* pb, int r, int K, int N,
                                       int64_t na, int64_t nb) {
  using C = Cfg<R>;
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

template <int R, bool kFp16>
cudaError_t launch(const AdapterArgs& p, cudaStream_t st) {
  auto kern = adapter_tc_kernel<R, kFp16>;
  cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), Cfg<R>::kBytes);
  if (e != cudaSuccess) return e;
  const int clusters = (p.T + p.cut.rows - 1) / p.cut.rows + (p.n + 1 < p.T ? p.n + 1 : p.T);
  return launch_pdl_clusters(kern, dim3(clusters * p.cut.ctas), dim3(kThreads), p.cut.ctas, Cfg<R>::kBytes, st, p);
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

// The most CTAs, up to two an SM (one above rank 64: all that run at a time; a cluster more waits for the first to end, 96 us instead of 63 at
// 8195 rows), from tiles of 128 or 64 rows and clusters of 8 to 1.  The slots' rows are unknown here: half a tile is
// lost to each slot, and a slot that is used has one at least.
AdapterCut adapter_cut(int T, int n, int rpad, int num_sms) {
  const int64_t fit = (rpad <= 64 ? 2 : 1) * num_sms;
  const int used = n < T ? n : T;
  AdapterCut best{kRows, 1};
  int64_t most = 0;
  for (int rows = kRows; rows >= kAdapterTileMin; rows /= 2) {
    const int64_t cut = static_cast<int64_t>(T) / rows + used / 2 + 1, tiles = cut > used ? cut : used;
    for (int c = 8; c >= 1; --c)
      if (tiles * c <= fit && tiles * c > most) most = tiles * c, best = AdapterCut{rows, c};
  }
  return best;
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
