// Routing rules other than a softmax over the chosen experts, by one warp a token:
//
//   s = sigmoid(z) or softmax(z) over all experts,  c = s + bias
//   the top_group groups of E / n_group neighbouring experts with the largest sum
//   of their best two c; of these groups' experts the k with the largest c (ties to
//   the lower group, the lower expert); gates = scale * s, over their sum or not
//
// (The bias only moves the choice, as for balance without an auxiliary
// loss. A NaN among the logits ranks below every number and counts in neither a
// softmax nor a group's sum; infinite logits have the scores' limits.)
#pragma once

#include "routing.cuh"

namespace fw {
namespace dev {

// Lane l holds experts MPL l .. MPL l + MPL - 1 (4, or 8 with more than 128): a group is
// then, as a rule, whole lanes, and its logits come with one load. (With experts 32
// apart in a lane every group took two reductions over the warp: one token of 7168,
// 256 experts in 8 groups, 10.2 us with the logits, this 9.1; 16 tokens 38.5 and 27.4.)

// s of this lane's experts, from their logits.
template <int MPL>
__device__ __forceinline__ void rule_scores(const float (&zl)[MPL], int E, int lane, bool sigmoid, float (&s)[MPL]) {
  if (sigmoid) {
#pragma unroll
    for (int m = 0; m < MPL; ++m) s[m] = 1.0f / (1.0f + expf(-zl[m]));
    return;
  }
  float top = -INFINITY;
#pragma unroll
  for (int m = 0; m < MPL; ++m) top = MPL * lane + m < E ? fmaxf(top, zl[m]) : top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  float sum = 0.f;
#pragma unroll
  for (int m = 0; m < MPL; ++m) {
    // (e^0, also where the difference of infinite logits is none; a NaN stays one, and out of the sum)
    s[m] = MPL * lane + m < E ? zl[m] == top ? 1.f : expf(zl[m] - top) : 0.f;
    sum += s[m] == s[m] ? s[m] : 0.f;
  }
  sum = warp_sum(sum);
#pragma unroll
  for (int m = 0; m < MPL; ++m) s[m] = s[m] / sum;
}

// (second: 0 where there is none, 1 where it is a NaN)
__device__ __forceinline__ uint32_t group_key(uint32_t top, uint32_t second) {
  return topk_key(second > 1u ? topk_value(top) + topk_value(second) : topk_value(top));
}

// The groups' choice: keys of experts in groups left out become 0. A group's best two
// keys (0 where there is no second) over the lanes that are the group, or, where its
// size is not a power of two of lanes, over the warp with the others' keys masked.
template <int MPL>
__device__ __forceinline__ void rule_groups(uint32_t (&key)[MPL], int E, int lane, const RouteRule& rule) {
  const int size = E / rule.n_group, lanes = size / MPL;
  if (size % MPL == 0 && (lanes & (lanes - 1)) == 0) {
    uint32_t best = 0, next = 0;
#pragma unroll
    for (int m = 0; m < MPL; ++m) {
      next = ::max(next, ::min(best, key[m]));
      best = ::max(best, key[m]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, best, o), other_next = __shfl_xor_sync(0xFFFFFFFFu, next, o);
      next = ::max(::min(best, other), ::max(next, other_next));
      best = ::max(best, other);
    }
    const uint32_t mine = group_key(best, next);
    int before = 0;
    for (int g = 0; g < rule.n_group; ++g) {
      const uint32_t other = __shfl_sync(0xFFFFFFFFu, mine, g * lanes);
      before += other > mine || (other == mine && (g + 1) * lanes <= lane);
    }
#pragma unroll
    for (int m = 0; m < MPL; ++m)
      if (before >= rule.top_group) key[m] = 0u;
    return;
  }
  const uint32_t per = (65536u + size - 1) / size;  // e / size = e per >> 16 for e < 256
  int group[MPL];
#pragma unroll
  for (int m = 0; m < MPL; ++m) group[m] = (int)((uint32_t)(MPL * lane + m) * per >> 16);
  uint32_t mine = 0;
  for (int g = 0; g < rule.n_group; ++g) {
    uint32_t best = 0, next = 0;  // this lane's best two keys of the group
#pragma unroll
    for (int m = 0; m < MPL; ++m) {
      const uint32_t v = group[m] == g ? key[m] : 0u;
      next = ::max(next, ::min(best, v));
      best = ::max(best, v);
    }
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    // one lane that holds it gives its next; of several that do, the others' best is as large
    const int from = __ffs(__ballot_sync(0xFFFFFFFFu, best == top)) - 1;
    const uint32_t second = __reduce_max_sync(0xFFFFFFFFu, lane == from ? next : best);
    if (lane == g) mine = group_key(top, second);
  }
  int before = 0;
  for (int g = 0; g < rule.n_group; ++g) {
    const uint32_t other = __shfl_sync(0xFFFFFFFFu, mine, g);
    before += other > mine || (other == mine && g < lane);
  }
  const uint32_t kept = __ballot_sync(0xFFFFFFFFu, lane < rule.n_group && before < rule.top_group);
#pragma unroll
  for (int m = 0; m < MPL; ++m)
    if (!(kept >> (group[m] & 31) & 1u)) key[m] = 0u;
}

// This lane's values of a row of E, experts MPL lane and on; past its end `none`. One load
// where E is a multiple of MPL (rows are then aligned to one).
template <int MPL>
__device__ __forceinline__ void load_mine(const float* row, int lane, int E, float none, float (&v)[MPL]) {
  const int e0 = MPL * lane;
  if (E % MPL == 0) {
    const float* at = row + (e0 < E ? e0 : 0);
    if constexpr (MPL == 8)  // (from L2: the logits may be of this kernel's other CTAs)
      asm volatile("ld.relaxed.gpu.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                   : "l"(at)
                   : "memory");
    else
      asm volatile("ld.relaxed.gpu.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(at) : "memory");
#pragma unroll
    for (int m = 0; m < MPL; ++m) v[m] = e0 < E ? v[m] : none;
  } else {
#pragma unroll
    for (int m = 0; m < MPL; ++m) v[m] = e0 + m < E ? __ldcg(row + e0 + m) : none;
  }
}

// load(z): the logits of this lane's experts, -infinity past the last one.
template <int MPL, class Load>
__device__ __forceinline__ void warp_rule_n(const Load& load, int E, int k, int lane, const RouteRule& rule, int* out_id, float* out_gate) {
  float zl[MPL], bias[MPL], s[MPL];
  load_mine<MPL>(rule.bias, lane, E, 0.f, bias);
  load(zl);
  rule_scores<MPL>(zl, E, lane, rule.score == kScoreSigmoid, s);
  uint32_t key[MPL];  // 0 past E and once chosen; at least 1 otherwise
#pragma unroll
  for (int m = 0; m < MPL; ++m) key[m] = MPL * lane + m < E ? topk_key(s[m] + bias[m]) : 0u;
  if (rule.n_group > 1) rule_groups<MPL>(key, E, lane, rule);
  int id = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int m = 1; m < MPL; ++m) best = ::max(best, key[m]);
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    uint32_t cand = 0xFFFFFFFFu;
#pragma unroll
    for (int m = MPL - 1; m >= 0; --m) cand = key[m] == top ? (uint32_t)(MPL * lane + m) : cand;
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, cand);
    if (lane == j) id = (int)e;
#pragma unroll
    for (int m = 0; m < MPL; ++m) key[m] = (uint32_t)(MPL * lane + m) == e ? 0u : key[m];
  }
  float w = 0.f;
#pragma unroll
  for (int m = 0; m < MPL; ++m) {
    const float v = __shfl_sync(0xFFFFFFFFu, s[m], (id / MPL) & 31);
    w = id % MPL == m ? v : w;
  }
  if (rule.renorm) w = w / (warp_sum(lane < k ? w : 0.f) + 1e-20f);
  *out_id = id;
  *out_gate = w * rule.scale;
}

// Lane j < k ends with (id_j, gate_j) of a token.
template <class Load>
__device__ __forceinline__ void warp_rule(const Load& load, int E, int k, int lane, const RouteRule& rule, int* out_id, float* out_gate) {
  if (E <= 128)
    warp_rule_n<4>(load, E, k, lane, rule, out_id, out_gate);
  else
    warp_rule_n<8>(load, E, k, lane, rule, out_id, out_gate);
}

// The counterparts of route_in_smem and route_one_in_smem under a rule; the gates are made with the choice.
template <int NT>
__device__ void route_in_smem_by_rule(const float* logits, int T, int E, int k, int S, const RouteRule& rule, SmemRouting& r) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < E + S; i += NT) r.mask[i] = 0;
  __syncthreads();
  for (int t = warp; t < T; t += NT / 32) {
    const auto load = [&](auto& z) { load_mine(logits + t * E, lane, E, -INFINITY, z); };
    float gate;
    int id;
    warp_rule(load, E, k, lane, rule, &id, &gate);
    if (lane < k) {
      r.ids[t * k + lane] = id;
      r.gates[t * k + lane] = gate;
      atomicOr(&r.mask[id], 1u << t);
    }
  }
  __syncthreads();
  if (warp == 0) group_in_smem(T, E, k, S, r, lane);
  __syncthreads();
}

template <int NT>
__device__ void route_one_in_smem_by_rule(const float* logits, int E, int k, int S, const RouteRule& rule, SmemRouting& r) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    const auto load = [&](auto& z) { load_mine(logits, lane, E, -INFINITY, z); };
    float gate;
    int id;
    warp_rule(load, E, k, lane, rule, &id, &gate);
    if (lane < k) r.gates[lane] = gate;
    if (S && lane == 0) r.gates[k] = 1.0f;
    group_one_in_smem(id, E, k, S, r, lane);
  }
  __syncthreads();
}

}  // namespace dev
}  // namespace fw
