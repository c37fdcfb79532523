// Scored selection of one token's experts by one warp (moe_plan_set_routing): softmax or sigmoid
// scores, a bias that only selects, expert groups, top-k, renormalised and scaled weights.  Shared by
// the routing kernels of route.cu in the place of topk_select.
//
//     s_e = sigmoid(l_e) or softmax(l)_e;   key_e = s_e + b_e,  key_e = -inf where l_e = -inf
//     groups of E / G consecutive experts: rank them by the sum of their `top` (1 or 2) largest keys,
//       keep the `keep` best, key_e = -inf in the others
//     the k largest keys, in order;  w = s (0 where the key is -inf);  w / (sum w + 1e-20) if renorm;
//       times scale
// Every order is the total order of rank_key: larger first, lower index on ties, NaN below -inf.  All in
// fp32 with expf and correctly rounded reciprocals: the scores are within a few units in the last place.
#pragma once

#include "topk.cuh"

namespace moe {

template <int PL>
MOE_DEVICE int score_select(const float (&v)[PL], int t, int E, int k, int32_t* __restrict__ ids,
                            float* __restrict__ gates, uint32_t* err, const ScoreArgs& sa) {
  const int lane = threadIdx.x & 31;
  constexpr float kInf = __builtin_huge_valf();
  // scores
  float s[PL];
  if (sa.sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = __frcp_rn(1.0f + expf(-v[i]));
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
    const float r = sum > 0.f ? __frcp_rn(sum) : (sum != sum ? sum : 0.f);
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] *= r;
  }
  // keys (rank_key order): 1 a padding lane, 2 NaN, above them the values
  uint32_t key[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 32 * i;
    key[i] = 1u;
    if (e < E) key[i] = rank_key(v[i] == -kInf ? -kInf : (sa.bias ? s[i] + sa.bias[e] : s[i]));
  }
  if (sa.groups > 1) {
    const int per = E / sa.groups;
    uint32_t mine = 0u;  // lane g: the ordered key of group g's score
    for (int g = 0; g < sa.groups; ++g) {
      const int lo = g * per, hi = lo + per;
      uint32_t b1 = 0u, b2 = 0u;  // this lane's two best keys of the group
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const int e = lane + 32 * i;
        const uint32_t c = (e >= lo && e < hi) ? key[i] : 0u;
        b2 = max(b2, min(b1, c));
        b1 = max(b1, c);
      }
      const uint32_t m1 = __reduce_max_sync(0xffffffffu, b1);
      float gs = rank_value(m1);
      if (sa.top == 2) {
        // one lane that holds the best gives its second instead
        const uint32_t who = __ballot_sync(0xffffffffu, b1 == m1);
        const uint32_t c = lane == __ffs(who) - 1 ? b2 : b1;
        gs += rank_value(__reduce_max_sync(0xffffffffu, c));
      }
      if (lane == g) mine = rank_key(gs);
    }
    int rank = 0;
    for (int g = 0; g < sa.groups; ++g) {
      const uint32_t o = __shfl_sync(0xffffffffu, mine, g);
      rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, lane < sa.groups && rank < sa.keep);
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !((kept >> (e / per)) & 1u)) key[i] = rank_key(-kInf);
    }
  }
  // the k largest keys
  int sel_e = 0;
  uint32_t sel_key = 0u;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < PL; ++i) {
      const bool gt = key[i] > best;  // strict: the lowest index keeps a tie
      best = gt ? key[i] : best;
      bi = gt ? i : bi;
    }
    const uint32_t win_key = __reduce_max_sync(0xffffffffu, best);
    const uint32_t cand = best == win_key ? static_cast<uint32_t>(lane + 32 * bi) : 0xffffffffu;
    const int win_e = static_cast<int>(__reduce_min_sync(0xffffffffu, cand));
    const bool owner = (win_e & 31) == lane;
#pragma unroll
    for (int i = 0; i < PL; ++i) key[i] = (owner && i == bi) ? 0u : key[i];
    if (lane == j) {
      sel_e = win_e;
      sel_key = win_key;
    }
  }
  float w = 0.f, l = 0.f;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const float si = __shfl_sync(0xffffffffu, s[i], sel_e & 31);
    const float li = __shfl_sync(0xffffffffu, v[i], sel_e & 31);
    if (i == (sel_e >> 5)) w = si, l = li;
  }
  if (lane >= k || sel_key == rank_key(-kInf)) w = 0.f;
  if (sa.renorm) {
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = __fdiv_rn(w, sum + 1e-20f);
  }
  const bool bad = lane < k && (l != l || l == kInf);
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_error(err, MOE_DEVERR_NONFINITE);
  if (lane < k) {
    ids[static_cast<size_t>(t) * k + lane] = sel_e;
    gates[static_cast<size_t>(t) * k + lane] = w * sa.scale;
  }
  return sel_e;
}

// The selection of a routing kernel: scored, or the softmax of the k largest logits.
template <int PL, bool kScored>
MOE_DEVICE int select_token(const float (&v)[PL], int t, int E, int k, int32_t* __restrict__ ids,
                            float* __restrict__ gates, uint32_t* err, const ScoreArgs& sa) {
  if (kScored) return score_select<PL>(v, t, E, k, ids, gates, err, sa);
  return topk_select<PL>(v, t, E, k, ids, gates, err);
}

}  // namespace moe
