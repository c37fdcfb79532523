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
// pair of fp32 values (its rounding error is kept), a lane's sum likewise (some 48 bits), joined in fp64.
// fp64 throughout would take six times as long as the memory on this chip (2 additions a clock and SM);
// the pair costs some 18 fp32 operations an element, half the memory's time.
#include "abi_checks.h"
#include "cluster.cuh"
#include "elems.cuh"

using namespace moe;

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kCluster = 8;   // CTAs of a request
constexpr int kGroups = 4;    // groups of 32 vectors whose loads are in flight together

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
};

// A probability as it counts: 0 unless 0 < v <= 2^64 (NaN, infinities and negative values count as 0; the
// bound keeps every sum of 2^30 of them finite).
MOE_DEVICE float clean(float v) {
  return __float_as_uint(v) - 1u < 0x5f800000u ? v : 0.0f;
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
  static MOE_DEVICE void load(const E* row, int first, int V, bool whole, float (&o)[kVec]) {
    if (whole) {
      alignas(16) E e[kVec];
      *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(row + first);
#pragma unroll
      for (int i = 0; i < kVec; ++i) o[i] = e[i].f32();
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) o[i] = first + i >= 0 && first + i < V ? row[first + i].f32() : 0.0f;
    }
  }
  // the cleaned values of vector v (zeros for v at or past `end`)
  MOE_DEVICE void get(int v, int end, float (&a)[kVec], float (&b)[kVec]) const {
    const int first = v * kVec - skip;
    const bool in = v < end, whole = in && together && first >= 0 && first + kVec <= V;
    if (in) {
      load(p, first, V, whole, a);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) a[i] = 0.0f;
    }
    if (in && q) {
      load(q, first, V, whole, b);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) b[i] = 0.0f;
    }
    if (static_cast<uint32_t>(drop - first) < kVec && drop >= 0) {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (first + i == drop) a[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) a[i] = clean(a[i]), b[i] = clean(b[i]);
  }
};

// hi + lo += max(p - q, 0), the rounding errors of the difference and of the sum kept in lo
MOE_DEVICE void add_rest(float p, float q, float& hi, float& lo) {
  const float d = p - q;
  const float bb = p - d;                       // (Knuth's two-sum of p and -q)
  const float ed = (p - (d + bb)) + (bb - q);
  const bool pos = d > 0.0f;
  const float v = pos ? d : 0.0f, e = pos ? ed : 0.0f;
  const float s = hi + v;
  const float t = s - hi;
  const float es = (hi - (s - t)) + (v - t);
  hi = s;
  lo += e + es;
}

MOE_DEVICE double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
MOE_DEVICE double warp_scan(double v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// The sum of the warp's range [v0, v1) of vectors.
template <typename E>
MOE_DEVICE double range_sum(const RowPair<E>& r, int v0, int v1, int lane) {
  constexpr int n = RowPair<E>::kVec;
  float hi = 0.0f, lo = 0.0f;
  for (int v = v0; v < v1; v += 32 * kGroups) {
    float a[kGroups][n], b[kGroups][n];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) r.get(v + 32 * g + lane, v1, a[g], b[g]);
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
      for (int i = 0; i < n; ++i) add_rest(a[g][i], b[g][i], hi, lo);
  }
  return warp_sum(static_cast<double>(hi) + static_cast<double>(lo));
}

// The lowest index of the range whose cumulative sum exceeds `at`; the last with a value above 0 where
// rounding leaves none.
template <typename E>
MOE_DEVICE int range_find(const RowPair<E>& r, int v0, int v1, int lane, double at) {
  constexpr int n = RowPair<E>::kVec;
  double before = 0.0;
  int last = -1;
  for (int v = v0; v < v1; v += 32) {
    float a[n], b[n];
    r.get(v + lane, v1, a, b);
    double own = 0.0;
    int mine = -1;
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (a[i] > b[i]) own += static_cast<double>(a[i]) - static_cast<double>(b[i]), mine = i;
    const double upto = before + warp_scan(own, lane);
    const uint32_t over = __ballot_sync(0xffffffffu, mine >= 0 && upto > at);
    if (over) {
      const int l = __ffs(over) - 1;
      double c = upto - own;
      int found = mine;
#pragma unroll
      for (int i = n - 1; i >= 0; --i) {  // (from the back: the lowest index stays)
        double s = c;
#pragma unroll
        for (int j = 0; j <= i; ++j)
          if (a[j] > b[j]) s += static_cast<double>(a[j]) - static_cast<double>(b[j]);
        if (a[i] > b[i] && s > at) found = i;
      }
      return __shfl_sync(0xffffffffu, (v + lane) * n - r.skip + found, l);
    }
    const uint32_t some = __ballot_sync(0xffffffffu, mine >= 0);
    if (some) last = __shfl_sync(0xffffffffu, (v + lane) * n - r.skip + mine, 31 - __clz(some));
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
  return last;
}

template <typename E>
__global__ void __launch_bounds__(kWarps * 32) verify_kernel(const VerifyArgs a) {
  __shared__ int s_refused;
  __shared__ double s_sum[kWarps];
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
    const int total = r.vectors(), parts = kCluster * kWarps;
    const int per = ((total + parts - 1) / parts + 31) / 32 * 32;
    const int part = rank * kWarps + warp;
    const int v0 = static_cast<int>(min(static_cast<int64_t>(part) * per, static_cast<int64_t>(total)));
    const int v1 = min(v0 + per, total);
    const double mine = range_sum(r, v0, v1, lane);
    if (lane == 0) s_sum[warp] = mine;
    cluster_barrier();
    // every warp: the ranges' sums in order, two a lane
    static_assert(kCluster * kWarps == 64, "two ranges a lane");
    const double s0 = ld_cluster_f64(cluster_addr(&s_sum[(2 * lane) % kWarps], 2 * lane / kWarps));
    const double s1 = ld_cluster_f64(cluster_addr(&s_sum[(2 * lane + 1) % kWarps], 2 * lane / kWarps));
    cluster_barrier();  // (the sums are read: the next round, or the exit, may follow)
    const double upto = warp_scan(s0 + s1, lane);
    const double sum = __shfl_sync(0xffffffffu, upto, 31);
    if (sum > 0.0) {
      const double at = us > 0.0f ? static_cast<double>(us) * sum : 0.0;
      // the first range that reaches past `at`, else the last that holds anything
      const double c0 = upto - s1, c1 = upto;
      uint32_t h0 = __ballot_sync(0xffffffffu, s0 > 0.0 && c0 > at), h1 = __ballot_sync(0xffffffffu, s1 > 0.0 && c1 > at);
      int found;
      if (h0 | h1) {
        const int l = __ffs(h0 | h1) - 1;
        found = 2 * l + ((h0 >> l) & 1u ? 0 : 1);
      } else {
        h0 = __ballot_sync(0xffffffffu, s0 > 0.0), h1 = __ballot_sync(0xffffffffu, s1 > 0.0);
        const int l = 31 - __clz(h0 | h1);
        found = 2 * l + ((h1 >> l) & 1u);
      }
      if (found == part) {
        const double x0 = __shfl_sync(0xffffffffu, upto - s1 - s0, found / 2);
        const double x1 = __shfl_sync(0xffffffffu, upto - s1, found / 2);
        const int tok = range_find(r, v0, v1, lane, at - (found & 1 ? x1 : x0));
        if (lane == 0) a.tokens[row] = tok;
      }
      return;
    }
    if (!refused || round) break;
    r.open(prow, nullptr, a.V, -1);  // nothing is left of p - q: from p itself
  }
  if (rank == 0 && threadIdx.x == 0) a.tokens[row] = -1;  // p holds nothing either
}

template <typename E>
cudaError_t launch(const VerifyArgs& a, int B, cudaStream_t st) {
  return launch_pdl_clusters(verify_kernel<E>, dim3(kCluster, B), dim3(kWarps * 32), kCluster, 0, st, a);
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
  LIN_TRY(dtype == MOE_BF16 ? launch<Bf16>(a, B, st) : dtype == MOE_FP16 ? launch<Fp16>(a, B, st) : launch<Fp32>(a, B, st));
  return MOE_OK;
}
