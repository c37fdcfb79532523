// Verification of drafted tokens (include/moe.h: moe_verify_drafts).
//
// A request's rows lo .. hi - 1 hold the target's probabilities p; row lo + i verifies draft i while
// u_i q_i < p_i.  Behind the first refusal one token is drawn from r = max(p - q, 0) of that row (of p
// behind the last draft): the lowest index whose cumulative sum of r exceeds u * S, S the total.
//
// Bound by memory: one row of p and one of q a request; the accepted rows cost one element each.  A
// cluster of CTAs shares a request: every CTA repeats the short acceptance test (two dependent loads;
// passing its answer on would take longer), then the row is cut into one contiguous range a warp.  Range
// sums meet in distributed shared memory, where every CTA finds the range that holds u * S; the warp that
// owns it goes through its range again (from L2) and writes the token.
//
// The answer is an index, so the sums are held far below the rows' resolution: p - q as an unevaluated
// pair of fp32 values (its rounding error is kept), every sum likewise (some 47 bits).
// fp64 would take six times as long as the memory on this chip (2 additions a clock and SM), and even its use in the
// reductions alone took a third of the time (24 warps an SM, 30 operations each); only the warp that writes the token
// uses it.  The elements' pairs go two elements an instruction (f32x2): some 10 instructions an element.
#include "abi_checks.h"
#include "cluster.cuh"
#include "elems.cuh"

using namespace moe;

namespace moe {
namespace {

constexpr int kClusterMax = 8;  // CTAs of a request
constexpr int kMarks = 4;       // partial sums of a range that are kept
constexpr int kGroups = 4;      // vectors whose loads are in flight together in the search
// vector pairs that a lane has in flight: with one CTA an SM (few requests) a range of 131072 / 64 values stays there whole
constexpr int ring_of(int blocks) { return blocks == 1 ? 16 : 8; }

struct VerifyArgs {
  const void* p = nullptr;
  const void* q = nullptr;  // or NULL: the draft is certain of its token
  int64_t ldp = 0, ldq = 0;
  const int32_t* drafts = nullptr;
  const int32_t* offsets = nullptr;
  const float* u = nullptr;
  const float* u_sample = nullptr;
  int32_t* tokens = nullptr;
  int32_t* accepted = nullptr;
  int R = 0, V = 0;
  int ctas = 1;  // of a cluster
};

// A probability as it counts: 0 unless 0 < v <= 2^64 (NaN, infinities and negative values count as 0; the
// bound keeps every sum of 2^30 of them finite).
constexpr uint32_t kLargest = 0x5f800000u;
MOE_DEVICE float clean(float v) {
  return __float_as_uint(v) - 1u < kLargest ? v : 0.0f;
}

// One row pair as the sums read it: vectors of 16 bytes from the first aligned address at or below the
// row's start.  Element i of vector v has the index v * kVec - skip + i; elements outside [0, V) count as 0.
template <typename E>
struct RowPair {
  static constexpr int kVec = 16 / sizeof(E);
  const E* p;
  const E* q;      // or nullptr
  int V, skip;     // skip: elements of the first vector that lie before the row
  int drop;        // an index whose p counts as 0 (the refused draft without draft probabilities), or -1
  bool together;   // p and q are aligned alike (else every element is loaded by itself)

  MOE_DEVICE void open(const E* p_, const E* q_, int V_, int drop_) {
    p = p_, q = q_, V = V_, drop = drop_;
    const uint32_t mp = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
    const uint32_t mq = q ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q) & 15u) : mp;
    skip = mp / sizeof(E);
    together = mp == mq;
  }
  MOE_DEVICE int vectors() const { return (V + skip + kVec - 1) / kVec; }
  static MOE_DEVICE uint4 load(const E* row, int first, int V, bool whole) {
    if (whole) return *reinterpret_cast<const uint4*>(row + first);
    alignas(16) E e[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) e[i] = first + i >= 0 && first + i < V ? row[first + i] : E{};
    return *reinterpret_cast<const uint4*>(e);
  }
  // vector v as it lies in memory (zeros at or past `end`)
  MOE_DEVICE void get(int v, int end, uint4& a, uint4& b) const {
    const int first = v * kVec - skip;
    const bool in = v < end, whole = together && first >= 0 && first + kVec <= V;
    a = in ? load(p, first, V, whole) : make_uint4(0u, 0u, 0u, 0u);
    b = in && q ? load(q, first, V, whole) : make_uint4(0u, 0u, 0u, 0u);
  }
  // its values as they count, with p raised to q where it is below: p - q is then max(p - q, 0)
  MOE_DEVICE void values(int v, const uint4& ra, const uint4& rb, float (&a)[kVec], float (&b)[kVec]) const {
    to_floats(ra, a);
    to_floats(rb, b);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) most = max(most, max(__float_as_uint(a[i]), __float_as_uint(b[i])));
    if (most > kLargest) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) a[i] = clean(a[i]), b[i] = clean(b[i]);
    }
    const int first = v * kVec - skip;
    if (drop >= first && drop < first + kVec) {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (first + i == drop) a[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) a[i] = fmaxf(a[i], b[i]);
  }
  static MOE_DEVICE void to_floats(const uint4& r, float (&o)[kVec]) {
    if constexpr (kVec == 8) {
      Raw8<E> x;
      x.a = r;
      x.to_f32(o);
    } else {
      o[0] = __uint_as_float(r.x), o[1] = __uint_as_float(r.y), o[2] = __uint_as_float(r.z), o[3] = __uint_as_float(r.w);
    }
  }
};

// Two fp32 values an instruction, each rounded as by itself.
struct Pair {
  uint64_t v;
  MOE_DEVICE Pair() {}
  MOE_DEVICE Pair(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
  MOE_DEVICE void get(float& x, float& y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
};
MOE_DEVICE Pair operator+(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
MOE_DEVICE Pair operator-(Pair a, Pair b) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(b.v), "l"(Pair(-1.0f, -1.0f).v), "l"(a.v));
  return r;
}

// hi + lo += p - q for two elements with p >= q, the rounding errors of the difference and of the sum kept in lo
// (Knuth's two-sum, twice)
MOE_DEVICE void add_rest(Pair p, Pair q, Pair& hi, Pair& lo) {
  const Pair d = p - q, bb = p - d;
  const Pair ed = (p - (d + bb)) + (bb - q);
  const Pair s = hi + d, t = s - hi;
  const Pair es = (hi - (s - t)) + (d - t);
  hi = s;
  lo = lo + (ed + es);
}

// hi + lo += v
MOE_DEVICE void add_value(Pair v, Pair& hi, Pair& lo) {
  const Pair s = hi + v, t = s - hi;
  lo = lo + ((hi - (s - t)) + (v - t));
  hi = s;
}

// hi + lo, |lo| <= half a step of hi: sums with some 47 bits at fp32's rate.
struct alignas(8) Wide {
  float hi, lo;
};
MOE_DEVICE Wide renormalised(float hi, float lo) {  // |hi| >= |lo|, or hi == 0
  const float s = hi + lo;
  return Wide{s, lo - (s - hi)};
}
MOE_DEVICE Wide operator+(Wide a, Wide b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  return renormalised(s, ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo));
}
MOE_DEVICE Wide operator*(float u, Wide a) {
  const float p = __fmul_rn(u, a.hi);  // (rounded here: fused into the sums below, its error would count twice)
  return renormalised(p, fmaf(u, a.hi, -p) + u * a.lo);
}
MOE_DEVICE bool operator>(Wide a, Wide b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

MOE_DEVICE Wide shfl(Wide v, int lane) {
  return Wide{__shfl_sync(0xffffffffu, v.hi, lane), __shfl_sync(0xffffffffu, v.lo, lane)};
}
MOE_DEVICE Wide warp_sum(Wide v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1)
    v = v + Wide{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
  return v;
}
MOE_DEVICE Wide warp_scan(Wide v, int lane) {  // inclusive
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const Wide n{__shfl_up_sync(0xffffffffu, v.hi, o), __shfl_up_sync(0xffffffffu, v.lo, o)};
    if (lane >= o) v = n + v;
  }
  return v;
}
MOE_DEVICE Wide operator-(Wide a, Wide b) { return a + Wide{-b.hi, -b.lo}; }
// p - q where p >= q, exactly
MOE_DEVICE Wide rest(float p, float q) {
  const float d = p - q, bb = p - d;
  return Wide{d, (p - (d + bb)) + (bb - q)};
}

// A lane's sum of rests.
struct Rest {
  Pair hi, lo;
  MOE_DEVICE Rest() : hi(0.0f, 0.0f), lo(0.0f, 0.0f) {}
  template <typename E>
  MOE_DEVICE void add(const RowPair<E>& r, int v, const uint4& a, const uint4& b) {
    constexpr int n = RowPair<E>::kVec;
    float x[n], y[n];
    r.values(v, a, b, x, y);
#pragma unroll
    for (int i = 0; i < n; i += 2) add_rest(Pair(x[i], x[i + 1]), Pair(y[i], y[i + 1]), hi, lo);
  }
  MOE_DEVICE Wide sum() const {
    float h0, h1, l0, l1;
    hi.get(h0, h1);
    lo.get(l0, l1);
    return renormalised(h0, l0) + renormalised(h1, l1);
  }
};

// The range's sum, the vectors v0 + lane, v0 + lane + 32, ... below v1 a lane.  The vectors come through a ring in shared
// memory (cp.async; a lane reads back what it copied, so no barrier): with loads into registers the warps waited for
// memory and for each other in turns, 20 GB/s a CTA.  marks[k][lane] is the lane's sum up to its vector (k + 1) * per_mark.
template <typename E, int kRing>
MOE_DEVICE Wide range_sum(const RowPair<E>& r, int v0, int v1, int lane, uint4* ring, Wide (*marks)[32], int per_mark) {
  const int n = (max(v1 - v0, 0) + 31) / 32;
  const auto ask = [&](int i) {
    const int v = v0 + 32 * i + lane, first = v * RowPair<E>::kVec - r.skip;
    uint4* at = ring + (i % kRing) * 64 + lane;
    if (v < v1 && r.together && first >= 0 && first + RowPair<E>::kVec <= r.V) {
      cp_async_16(smem_u32(at), r.p + first);
      if (r.q) cp_async_16(smem_u32(at + 32), r.q + first);
    } else {
      uint4 a, b;
      r.get(v, v1, a, b);
      at[0] = a, at[32] = b;
    }
    if (!r.q) at[32] = make_uint4(0u, 0u, 0u, 0u);
  };
#pragma unroll 1
  for (int i = 0; i < kRing - 1; ++i) {
    if (i < n) ask(i);
    cp_async_commit();
  }
  Rest sum;
  int mark = per_mark, k = 0;
  for (int i = 0; i < n; ++i) {
    if (i + kRing - 1 < n) ask(i + kRing - 1);
    cp_async_commit();
    cp_async_wait<kRing - 1>();
    const uint4* at = ring + (i % kRing) * 64 + lane;
    sum.add(r, v0 + 32 * i + lane, at[0], at[32]);
    if (i + 1 == mark && k < kMarks) marks[k++][lane] = sum.sum(), mark += per_mark;
  }
  cp_async_wait<0>();
  return sum.sum();
}

// The same for a range of whole vectors whose values are all in [0, 2) (plain probabilities) and that has no dropped
// index: no vector and no value is checked, which leaves some 11 instructions an element (of 36).  Returns whether the
// values were that, seen from the bits of all of them: a sign, or the exponents of 2 and more, NaN and infinity.
template <typename E, bool kQ, int kRing>
MOE_DEVICE bool range_sum_plain(const RowPair<E>& r, int v0, int n, int lane, uint4* ring, Wide (*marks)[32], int per_mark,
                                Wide& result) {
  constexpr int m = RowPair<E>::kVec;
  const E* p = r.p + (static_cast<int64_t>(v0 + lane) * m - r.skip);
  const E* q = kQ ? r.q + (static_cast<int64_t>(v0 + lane) * m - r.skip) : nullptr;
  const uint32_t base = smem_u32(ring + lane);
  uint32_t fill = 0, from = 0, bits = 0;
  const auto ask = [&] {
    cp_async_16(base + fill, p);
    if (kQ) cp_async_16(base + fill + 512, q);
    p += 32 * m;
    if (kQ) q += 32 * m;
    fill = (fill + 1024) & (1024 * kRing - 1);
  };
#pragma unroll 1
  for (int i = 0; i < kRing - 1; ++i) {
    if (i < n) ask();
    cp_async_commit();
  }
  Rest sum;
  int mark = per_mark, k = 0;
#pragma unroll 2
  for (int i = 0; i < n; ++i) {
    if (i + kRing - 1 < n) ask();
    cp_async_commit();
    cp_async_wait<kRing - 1>();
    const uint4* at = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(ring + lane) + from);
    from = (from + 1024) & (1024 * kRing - 1);
    float x[m], y[m];
    RowPair<E>::to_floats(at[0], x);
    if (kQ) RowPair<E>::to_floats(at[32], y);
#pragma unroll
    for (int j = 0; j < m; ++j) {
      bits |= __float_as_uint(x[j]);
      if (kQ) bits |= __float_as_uint(y[j]), x[j] = fmaxf(x[j], y[j]);
    }
#pragma unroll
    for (int j = 0; j < m; j += 2) {
      if (kQ)
        add_rest(Pair(x[j], x[j + 1]), Pair(y[j], y[j + 1]), sum.hi, sum.lo);
      else
        add_value(Pair(x[j], x[j + 1]), sum.hi, sum.lo);
    }
    if (i + 1 == mark && k < kMarks) marks[k++][lane] = sum.sum(), mark += per_mark;
  }
  cp_async_wait<0>();
  result = sum.sum();
  return !__any_sync(0xffffffffu, bits >> 30);
}

// The sum of the vectors [v0, v1), one lane's.
template <typename E>
MOE_DEVICE Wide lane_sum(const RowPair<E>& r, int v0, int v1) {
  Rest sum;
  for (int v = v0; v < v1; v += kGroups) {
    uint4 a[kGroups], b[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) r.get(v + g, v1, a[g], b[g]);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) sum.add(r, v + g, a[g], b[g]);
  }
  return sum.sum();
}

// The lowest index of the range [v0, v1) whose cumulative sum exceeds `at`; the last with a value above 0 where rounding
// leaves none.  ring: the range's vectors, group i of 32 at 64 i, or nullptr.
template <typename E>
MOE_DEVICE int range_find(const RowPair<E>& r, int v0, int v1, Wide at, const uint4* ring,
                                       const Wide (*marks)[32], int per_mark) {
  constexpr int n = RowPair<E>::kVec;
  const int lane = threadIdx.x & 31, start = v0, whole_end = v1;
  // the marked part that it lies in
  const int written = min((v1 - v0 + 31) / 32 / per_mark, kMarks);
  Wide before{0.0f, 0.0f};
  int k = 0;
#pragma unroll 1
  for (; k < written; ++k) {
    const Wide part = warp_sum(marks[k][lane]);
    if (part > at) break;
    before = part;
  }
  if (v0 + 32 * per_mark * k < v1) {
    v0 += 32 * per_mark * k;
    if (k < written) v1 = min(v0 + 32 * per_mark, v1);
    at = at - before;
  }
  // a long part: a lane's contiguous 32nd of it
  if (v1 - v0 > 32 * 16) {
    const int per = (v1 - v0 + 31) / 32, l0 = min(v0 + lane * per, v1), l1 = min(l0 + per, v1);
    const Wide own = lane_sum(r, l0, l1), upto = warp_scan(own, lane);
    const uint32_t over = __ballot_sync(0xffffffffu, own.hi > 0.0f && upto > at);
    if (over) {
      const int l = __ffs(over) - 1;
      at = at - shfl(upto - own, l);
      v0 = __shfl_sync(0xffffffffu, l0, l), v1 = __shfl_sync(0xffffffffu, l1, l);
      ring = nullptr;
    }
  }
#pragma unroll 1
  for (int v = v0; v < v1; v += 32) {
    uint4 ra, rb;
    if (ring)
      ra = ring[(v - start) * 2 + lane], rb = r.q ? ring[(v - start) * 2 + 32 + lane] : make_uint4(0u, 0u, 0u, 0u);
    else
      r.get(v + lane, v1, ra, rb);
    float a[n], b[n];
    r.values(v + lane, ra, rb, a, b);
    Wide own{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < n; ++i) own = own + rest(a[i], b[i]);
    const Wide upto = warp_scan(own, lane);
    const uint32_t over = __ballot_sync(0xffffffffu, own.hi > 0.0f && upto > at);
    if (over) {
      Wide c = upto - own;
      int found = -1, last = 0;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        c = c + rest(a[i], b[i]);
        if (a[i] > b[i]) {
          last = i;
          if (found < 0 && c > at) found = i;
        }
      }
      return __shfl_sync(0xffffffffu, (v + lane) * n - r.skip + (found < 0 ? last : found), __ffs(over) - 1);
    }
    at = at - shfl(upto, 31);
  }
  // none by rounding: the last value above 0 of the part, else of the range
  for (int again = 0;; ++again) {
    int last = -1;
    for (int v = v0; v < v1; v += 32) {
      uint4 ra, rb;
      float a[n], b[n];
      r.get(v + lane, v1, ra, rb);
      r.values(v + lane, ra, rb, a, b);
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (a[i] > b[i]) last = (v + lane) * n - r.skip + i;
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (last >= 0 || again) return last;
    v0 = start, v1 = whole_end;
  }
}

template <typename E, int W, int kBlocks>
__global__ void __launch_bounds__(W * 32, kBlocks) verify_kernel(const VerifyArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  constexpr int kRing = ring_of(kBlocks);
  uint4* ring = reinterpret_cast<uint4*>(smem_raw) + (threadIdx.x >> 5) * (kRing * 64);
  Wide (*marks)[32] = reinterpret_cast<Wide (*)[32]>(smem_raw + W * kRing * 64 * 16) + (threadIdx.x >> 5) * kMarks;
  __shared__ int s_refused;
  __shared__ Wide s_sum[W];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  const int lo = a.offsets[b], hi = a.offsets[b + 1];
  const bool valid = lo >= 0 && hi >= lo && hi <= a.R;
  if (!valid || hi == lo) {  // (the same for every CTA of the cluster)
    if (rank == 0 && threadIdx.x == 0) a.accepted[b] = valid ? 0 : -1;
    return;
  }
  // ---- acceptance: the first refused draft --------------------------------------------------------
  const int n = hi - lo - 1;
  if (threadIdx.x == 0) s_refused = n;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int64_t row = lo + i;
    const int tok = a.drafts[row];
    float p = 0.0f, q = 1.0f;
    if (tok >= 0 && tok < a.V) {
      p = clean((static_cast<const E*>(a.p) + row * a.ldp)[tok].f32());
      if (a.q) q = clean((static_cast<const E*>(a.q) + row * a.ldq)[tok].f32());
    }
    // (the product is exact in fp64: 24 + 24 bits)
    if (!(static_cast<double>(a.u[row]) * static_cast<double>(q) < static_cast<double>(p))) atomicMin(&s_refused, i);
  }
  __syncthreads();
  const int passed = s_refused;
  const int64_t row = lo + passed;
  if (rank == 0) {
    for (int i = threadIdx.x; i < hi - lo; i += blockDim.x)
      if (i != passed) a.tokens[lo + i] = i < passed ? a.drafts[lo + i] : -1;
    if (threadIdx.x == 0) a.accepted[b] = passed;
  }
  // ---- the token behind them ------------------------------------------------------------------------
  const float us = a.u_sample[b];
  RowPair<E> r;
  const E* prow = static_cast<const E*>(a.p) + row * a.ldp;
  const bool refused = passed < n;
  r.open(prow, refused && a.q ? static_cast<const E*>(a.q) + row * a.ldq : nullptr, a.V,
         refused && !a.q ? a.drafts[row] : -1);
  for (int round = 0;; ++round) {
    const int total = r.vectors(), parts = a.ctas * W;
    const int per = ((total + parts - 1) / parts + 31) / 32 * 32;
    const int part = rank * W + warp;
    const int v0 = static_cast<int>(min(static_cast<int64_t>(part) * per, static_cast<int64_t>(total)));
    const int v1 = min(v0 + per, total);
    const int per_mark = (per / 32 + kMarks) / (kMarks + 1);
    Wide mine;
    const int e0 = v0 * RowPair<E>::kVec - r.skip, e1 = v1 * RowPair<E>::kVec - r.skip;  // elements [e0, e1)
    bool done = false;
    if (r.together && e0 >= 0 && e1 <= a.V && (v1 - v0) % 32 == 0 && !(r.drop >= e0 && r.drop < e1))
      done = r.q ? range_sum_plain<E, true, kRing>(r, v0, (v1 - v0) / 32, lane, ring, marks, per_mark, mine)
                 : range_sum_plain<E, false, kRing>(r, v0, (v1 - v0) / 32, lane, ring, marks, per_mark, mine);
    if (!done) mine = range_sum<E, kRing>(r, v0, v1, lane, ring, marks, per_mark);
    mine = warp_sum(mine);
    if (lane == 0) s_sum[warp] = mine;
    cluster_barrier();
    // every warp: the ranges' sums in order, kPer neighbours a lane
    constexpr int kPer = kClusterMax * W / 32;
    static_assert(kPer >= 1 && W % kPer == 0, "a lane's ranges are one CTA's");
    Wide c[kPer], own{0.0f, 0.0f};  // c: cumulative within the lane
    uint32_t some = 0;
    if (kPer * lane < parts) {
      const uint32_t from = cluster_addr(&s_sum[kPer * lane % W], kPer * lane / W);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float2 v = ld_cluster_f32x2(from + i * sizeof(Wide));
        c[i] = Wide{v.x, v.y};
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) some |= c[i].hi > 0.0f ? 1u << i : 0u, own = own + c[i], c[i] = own;
    }
    cluster_arrive();  // the sums are read: the next round, or the exit, waits for all of that
    const Wide upto = warp_scan(own, lane), sum = shfl(upto, 31);
    if (sum.hi > 0.0f) {
      const Wide at = us > 0.0f ? us * sum : Wide{0.0f, 0.0f}, before = upto - own;
      // the first range that reaches past `at`, else the last that holds anything
      uint32_t over = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if ((some >> i & 1u) && before + c[i] > at) over |= 1u << i;
      const uint32_t lanes_over = __ballot_sync(0xffffffffu, over != 0), lanes_some = __ballot_sync(0xffffffffu, some != 0);
      const int l = lanes_over ? __ffs(lanes_over) - 1 : 31 - __clz(lanes_some);
      const int in = __shfl_sync(0xffffffffu, lanes_over ? __ffs(over) - 1 : 31 - __clz(some), l);
      const int found = kPer * l + in;
      if (found == part) {
        Wide skipped{0.0f, 0.0f};  // what lies before this range within the lane's
#pragma unroll
        for (int i = 0; i + 1 < kPer; ++i)
          if (i < in) skipped = c[i];
        const Wide left = at - shfl(before + skipped, l);
        __syncwarp();
        const int tok = range_find(r, v0, v1, left, (v1 - v0 + 31) / 32 <= kRing ? ring : nullptr, marks, per_mark);
        if (lane == 0) a.tokens[row] = tok;
      }
      cluster_wait();
      return;
    }
    cluster_wait();
    if (!refused || round) break;
    r.open(prow, nullptr, a.V, -1);  // nothing is left of p - q: from p itself
  }
  if (rank == 0 && threadIdx.x == 0) a.tokens[row] = -1;  // p holds nothing either
}

template <typename E, int W, int kBlocks>
cudaError_t launch_warps(VerifyArgs a, int B, int ctas, cudaStream_t st) {
  constexpr int smem = W * (ring_of(kBlocks) * 64 * 16 + kMarks * 32 * sizeof(Wide));
  cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(verify_kernel<E, W, kBlocks>), smem);
  if (e != cudaSuccess) return e;
  a.ctas = ctas;
  return launch_pdl_clusters(verify_kernel<E, W, kBlocks>, dim3(ctas, B), dim3(W * 32), ctas, smem, st, a);
}

template <typename E>
cudaError_t launch(const VerifyArgs& a, int B, int num_sms, cudaStream_t st) {
  // Few requests: the most threads a request, a CTA of 8 warps an SM (8 requests of 131072: 10.8 us, 12.8 with 4 warps).
  // Up to three such CTAs an SM, where a warp's range has three groups of 32 vectors at least (48 requests of 131072:
  // 17.0 us, with CTAs of 4 warps 19.6; of 32003: 9.1 and 12.1; of 16384, two groups: 7.6 and 7.3; 64 of 131072, which do
  // not all run at once: 23.5 and 23.1).
  // Many: CTAs of 4 warps, six an SM, whose acceptance, reading and search overlap (192 requests of 131072: 39 us, 46 with
  // 8), as long as a warp's range has three groups where all CTAs run at once (100 requests of 32003: 8 CTAs 10.4 us, 4
  // 13.5; six an SM do not always fit in clusters, so five and a half are counted: 114 of 16384, 4 CTAs 10.3, 2 9.6), eight
  // where they do not (192 requests of 32003: 4 CTAs 16.7 us, 8 18.2).
  const int groups = a.V / (32 * RowPair<E>::kVec);
  if (B * kClusterMax <= num_sms) return launch_warps<E, 8, 1>(a, B, kClusterMax, st);
  if (B * kClusterMax <= 3 * num_sms && groups >= 3 * 8 * kClusterMax) return launch_warps<E, 8, 3>(a, B, kClusterMax, st);
  int ctas = kClusterMax;
  while (ctas > 1 && groups < (B * ctas <= 11 * num_sms / 2 ? 3 : 8) * 4 * ctas) ctas /= 2;
  return launch_warps<E, 4, 6>(a, B, ctas, st);
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_verify_drafts(const void* target, moe_dtype dtype, int64_t ldt, const void* draft_probs,
                                        int64_t ldd, int R, int V, const int32_t* drafts, const int32_t* offsets, int B,
                                        const float* u, const float* u_sample, int32_t* tokens, int32_t* accepted,
                                        moe_stream_t stream) {
  if (R < 0 || V < 1 || B < 0) return bad(MOE_ERR_INVALID_ARG, "need R >= 0, V >= 1, B >= 0");
  if (!known(dtype)) return bad(MOE_ERR_INVALID_ARG, "unknown element type");
  if (V > (1 << 30) || B > 65535) return bad(MOE_ERR_UNSUPPORTED, "at most 2^30 tokens and 65535 requests");
  if (B == 0) return MOE_OK;
  if (!offsets || !u_sample || !accepted) return bad(MOE_ERR_INVALID_ARG, "offsets, u_sample and accepted are required");
  if (!aligned(drafts, 4) || !aligned(offsets, 4) || !aligned(u, 4) || !aligned(u_sample, 4) || !aligned(tokens, 4) ||
      !aligned(accepted, 4))
    return bad(MOE_ERR_INVALID_ARG, "drafts, offsets, u, u_sample, tokens and accepted must be aligned to their elements");
  if (R > 0) {
    if (!target || !drafts || !u || !tokens)
      return bad(MOE_ERR_INVALID_ARG, "target, drafts, u and tokens are required");
    if (ldt < V || (draft_probs && ldd < V)) return bad(MOE_ERR_INVALID_ARG, "a row pitch is below V");
    if (!aligned(target, elem_bytes(dtype)) || !aligned(draft_probs, elem_bytes(dtype)))
      return bad(MOE_ERR_INVALID_ARG, "probabilities must be aligned to their elements");
  }
  VerifyArgs a;
  a.p = target, a.ldp = ldt, a.q = draft_probs, a.ldq = ldd, a.R = R, a.V = V;
  a.drafts = drafts, a.offsets = offsets, a.u = u, a.u_sample = u_sample, a.tokens = tokens, a.accepted = accepted;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  LIN_TRY(dtype == MOE_BF16 ? launch<Bf16>(a, B, current_sms(), st) : dtype == MOE_FP16 ? launch<Fp16>(a, B, current_sms(), st)
                                                                     : launch<Fp32>(a, B, current_sms(), st));
  return MOE_OK;
}
