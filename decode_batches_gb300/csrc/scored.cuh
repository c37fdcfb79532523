// Scored selection of one token's experts by one warp (moe_plan_set_routing): softmax or sigmoid
// scores, a bias that only selects, expert groups, top-k, renormalised and scaled weights.  Shared by
// the routing kernels of route.cu in the place of topk_select.
//
//     s_e = sigmoid(l_e) or softmax(l)_e;   key_e = s_e + b_e,  key_e = -inf where l_e = -inf
//     groups of E / G consecutive experts: rank them by the sum of their `top` (1 or 2) largest keys,
//       keep the `keep` best, key_e = -inf in the others
//     the k largest keys, in order;  w = s (0 where the key is -inf);  w / (sum w + 1e-20) if renorm;
//       times scale
// A softmax over a NaN would make every score NaN, and masked experts, whose key is a number, would rank
// first.  So NaN logits keep a score of NaN of their own and stay out of the sum, +inf ones share the score
// 1 as in the limit, and the error bit says so whichever experts are chosen.
// Every order is the total order of rank_key: larger first, lower index on ties, NaN below -inf.  All in
// fp32 with expf (2 ulp) and reciprocals good to 1 ulp.  A sigmoid is within a few units in the last place;
// a softmax score besides by the rounding of its difference, |l - max| 2^-24 relative, and of the sum.
#pragma once

#include "topk.cuh"

namespace moe {

MOE_DEVICE float rcp_approx(float x) {  // 1 ulp
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// scr: E words of shared memory of this warp's own.  One token is a few hundred instructions of one
// warp, so what bounds the kernel is their number: a lane keeps its two best keys in registers (a
// rescan, under a warp-uniform branch, when both are taken), a group's members are divided over the
// lanes through scr, and the chosen scores are fetched through it.  Against rounds that rescan every
// key and groups reduced one after the other: E = 384, 12 groups, 8195 tokens 37 -> 22 us (in blocks of 16
// tokens; 15 in the blocks of 8 that route.cu takes).
template <int PL>
MOE_DEVICE int score_select(const float (&v)[PL], int t, int E, int k, int32_t* __restrict__ ids,
                            float* __restrict__ gates, uint32_t* err, const ScoreArgs& sa, uint32_t* scr) {
  const int lane = threadIdx.x & 31;
  constexpr float kInf = __builtin_huge_valf();
  // scores
  float s[PL];
  bool odd = false;  // some logit of the token is NaN or +inf
  if (sa.sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      s[i] = rcp_approx(1.0f + expf(-v[i]));
      odd |= lane + 32 * i < E && !(v[i] < kInf);
    }
    odd = __any_sync(0xffffffffu, odd);
  } else {
    float m = -kInf;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + 32 * i < E) m = fmaxf(m, v[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -kInf) m = 0.f;  // every expert masked: all scores 0
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      s[i] = lane + 32 * i < E ? expf(v[i] - m) : 0.f;
      sum += s[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    odd = sum != sum;  // exp(NaN), or inf - inf
    if (odd) {  // again without the NaN logits, inf - inf as 0
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        if (lane + 32 * i < E && v[i] == m) s[i] = 1.f;
        sum += s[i] == s[i] ? s[i] : 0.f;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    const float r = sum > 0.f ? __frcp_rn(sum) : 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] *= r;
  }
  // keys (rank_key order): 1 a padding lane, 2 NaN, above them the values
  const uint32_t none = rank_key(-kInf);
  uint32_t key[PL];
  if (!odd && !sa.bias) {  // scores are numbers >= 0: their bits are in order
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const uint32_t kk = v[i] == -kInf ? none : (__float_as_uint(s[i]) | 0x80000000u);
      key[i] = lane + 32 * i < E ? kk : 1u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      key[i] = 1u;
      if (e < E) key[i] = v[i] == -kInf ? none : rank_key(sa.bias ? s[i] + sa.bias[e] : s[i]);
    }
  }
  if (sa.groups > 1) {
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + 32 * i < E) scr[lane + 32 * i] = key[i];
    __syncwarp();
    // sa.lanes lanes take the members of a group in turn, starting at different places (banks)
    const int per = E / sa.groups, g = lane / sa.lanes, sub = lane % sa.lanes;
    uint32_t b1 = 0u, b2 = 0u;  // the lane's two best keys of the group
    if (g < sa.groups) {
      const int n = (per - sub + sa.lanes - 1) / sa.lanes;  // members sub, sub + lanes, ...
      int at = min(g, n - 1) * sa.lanes;
#pragma unroll 4
      for (int c = 0; c < n; ++c) {  // (n == 0: a group smaller than its lanes)
        const uint32_t kk = scr[g * per + sub + at];
        b2 = max(b2, min(b1, kk));
        b1 = max(b1, kk);
        at += sa.lanes;
        at = at < n * sa.lanes ? at : 0;
      }
    }
    for (int o = 1; o < sa.lanes; o <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
      b2 = max(min(b1, o1), max(b2, o2));
      b1 = max(b1, o1);
    }
    const uint32_t mine = rank_key(sa.top == 2 ? rank_value(b1) + rank_value(b2) : rank_value(b1));
    int rank = 0;
    for (int o = 0; o < sa.groups; ++o) {
      const uint32_t other = __shfl_sync(0xffffffffu, mine, o * sa.lanes);
      rank += (other > mine || (other == mine && o < g)) ? 1 : 0;
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, g < sa.groups && rank < sa.keep);
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      const uint32_t ge = (static_cast<uint32_t>(e) * sa.per_magic) >> 20;  // e / per
      if (e < E && !((kept >> (ge * sa.lanes)) & 1u)) key[i] = none;
    }
  }
  // the k largest keys: a lane offers its best; b1 / b2 its two best left, `left` how many of them
  uint32_t taken = 0u, b1, b2;
  int i1, i2, left;
  auto scan = [&]() {
    b1 = b2 = 0u, i1 = i2 = 0, left = 2;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const uint32_t kk = (taken >> i) & 1u ? 0u : key[i];
      const bool first = kk > b1, second = kk > b2;  // strict: the lowest index keeps a tie
      b2 = first ? b1 : (second ? kk : b2);
      i2 = first ? i1 : (second ? i : i2);
      b1 = first ? kk : b1;
      i1 = first ? i : i1;
    }
  };
  scan();
  int sel_e = 0;
  uint32_t sel_key = 0u;
  for (int j = 0; j < k; ++j) {
    const uint32_t win_key = __reduce_max_sync(0xffffffffu, b1);
    const uint32_t cand = b1 == win_key ? static_cast<uint32_t>(lane + 32 * i1) : 0xffffffffu;
    const int win_e = static_cast<int>(__reduce_min_sync(0xffffffffu, cand));
    if (lane == j) {
      sel_e = win_e;
      sel_key = win_key;
    }
    if (cand == static_cast<uint32_t>(win_e)) {
      taken |= 1u << i1;
      b1 = b2;
      i1 = i2;
      --left;
    }
    if (PL > 2 && __any_sync(0xffffffffu, left == 0)) {
      if (left == 0) scan();
    } else if (PL <= 2 && left == 0) {
      b1 = 0u;
    }
  }
  // the chosen experts' scores
  __syncwarp();
#pragma unroll
  for (int i = 0; i < PL; ++i)
    if (lane + 32 * i < E) scr[lane + 32 * i] = __float_as_uint(s[i]);
  __syncwarp();
  float w = lane < k && sel_key != none ? __uint_as_float(scr[sel_e]) : 0.f;
  if (sa.renorm) {
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = __fdiv_rn(w, sum + 1e-20f);
  }
  if (odd) {  // flagged: with sigmoid scores, which stand alone, if one of them was chosen
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const float li = __shfl_sync(0xffffffffu, v[i], sel_e & 31);
      if (i == (sel_e >> 5)) l = li;
    }
    if (__any_sync(0xffffffffu, !sa.sigmoid || (lane < k && !(l < kInf))) && lane == 0)
      set_error(err, MOE_DEVERR_NONFINITE);
  }
  if (lane < k) {
    ids[static_cast<size_t>(t) * k + lane] = sel_e;
    gates[static_cast<size_t>(t) * k + lane] = w * sa.scale;
  }
  return sel_e;
}

// The selection of a routing kernel: scored, or the softmax of the k largest logits.
template <int PL, bool kScored>
MOE_DEVICE int select_token(const float (&v)[PL], int t, int E, int k, int32_t* __restrict__ ids,
                            float* __restrict__ gates, uint32_t* err, const ScoreArgs& sa, uint32_t* scr) {
  if (kScored) return score_select<PL>(v, t, E, k, ids, gates, err, sa, scr);
  return topk_select<PL>(v, t, E, k, ids, gates, err);
}

}  // namespace moe
