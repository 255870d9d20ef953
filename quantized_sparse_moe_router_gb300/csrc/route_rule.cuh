// Routing rules other than a softmax over the chosen experts, by one warp a token:
//
//   s = sigmoid(z) or softmax(z) over all experts,  c = s + bias
//   the top_group groups of E / n_group neighbouring experts with the largest sum
//   of their best two c; of these groups' experts the k with the largest c (ties to
//   the lower group, the lower expert); gates = scale * s, over their sum or not
//
// (The bias only moves the choice: DeepSeek-style balance without an auxiliary
// loss. A NaN among the logits ranks below every number.)
#pragma once

#include "routing.cuh"

namespace fw {
namespace dev {

// s of this lane's experts (lane + 32 m), from their logits.
template <int MPL>
__device__ __forceinline__ void rule_scores(const float (&zl)[kMaxEPerLane], int E, int lane, bool sigmoid, float (&s)[MPL]) {
  if (sigmoid) {
#pragma unroll
    for (int m = 0; m < MPL; ++m) s[m] = 1.0f / (1.0f + expf(-zl[m]));
    return;
  }
  float top = -INFINITY;
#pragma unroll
  for (int m = 0; m < MPL; ++m) top = lane + 32 * m < E ? fmaxf(top, zl[m]) : top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  float sum = 0.f;
#pragma unroll
  for (int m = 0; m < MPL; ++m) {
    s[m] = lane + 32 * m < E ? expf(zl[m] - top) : 0.f;
    sum += s[m];
  }
  sum = warp_sum(sum);
#pragma unroll
  for (int m = 0; m < MPL; ++m) s[m] = s[m] / sum;
}

// The groups' choice: keys of experts in groups left out become 0. Group g's best
// key, then the best of the others in it, by integer warp reductions (as in
// warp_topk); lane g keeps the group's score, and ranks it against the others'.
template <int MPL>
__device__ __forceinline__ void rule_groups(uint32_t (&key)[MPL], int E, int lane, const RouteRule& rule) {
  const int size = E / rule.n_group;
  const uint32_t per = (65536u + size - 1) / size;  // e / size = e per >> 16 for e < 256
  int group[MPL];
#pragma unroll
  for (int m = 0; m < MPL; ++m) group[m] = (int)((uint32_t)(lane + 32 * m) * per >> 16);
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
    const float score = second ? topk_value(top) + topk_value(second) : topk_value(top);
    if (lane == g) mine = topk_key(score);
  }
  int before = 0;
  for (int g = 0; g < rule.n_group; ++g) {
    const uint32_t other = __shfl_sync(0xFFFFFFFFu, mine, g);
    before += other > mine || (other == mine && g < lane);
  }
  const uint32_t kept = __ballot_sync(0xFFFFFFFFu, lane < rule.n_group && before < rule.top_group);
#pragma unroll
  for (int m = 0; m < MPL; ++m)
    if (!(kept >> group[m] & 1u)) key[m] = 0u;
}

template <int MPL>
__device__ __forceinline__ void warp_rule_n(const float (&zl)[kMaxEPerLane], int E, int k, int lane, const RouteRule& rule, int* out_id, float* out_gate) {
  float s[MPL];
  rule_scores<MPL>(zl, E, lane, rule.score == kScoreSigmoid, s);
  uint32_t key[MPL];  // 0 past E and once chosen; at least 1 otherwise
#pragma unroll
  for (int m = 0; m < MPL; ++m) key[m] = lane + 32 * m < E ? topk_key(s[m] + __ldg(rule.bias + lane + 32 * m)) : 0u;
  if (rule.n_group > 1) rule_groups<MPL>(key, E, lane, rule);
  int id = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int m = 1; m < MPL; ++m) best = ::max(best, key[m]);
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    uint32_t cand = 0xFFFFFFFFu;
#pragma unroll
    for (int m = MPL - 1; m >= 0; --m) cand = key[m] == top ? (uint32_t)(lane + 32 * m) : cand;
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, cand);
    if (lane == j) id = (int)e;
#pragma unroll
    for (int m = 0; m < MPL; ++m) key[m] = (uint32_t)(lane + 32 * m) == e ? 0u : key[m];
  }
  float w = 0.f;
#pragma unroll
  for (int m = 0; m < MPL; ++m) {
    const float v = __shfl_sync(0xFFFFFFFFu, s[m], id & 31);
    w = id >> 5 == m ? v : w;
  }
  if (rule.renorm) w = w / (warp_sum(lane < k ? w : 0.f) + 1e-20f);
  *out_id = id;
  *out_gate = w * rule.scale;
}

// Lane j < k ends with (id_j, gate_j) of a token whose logits are z[lane + 32 m].
__device__ __forceinline__ void warp_rule(const float (&zl)[kMaxEPerLane], int E, int k, int lane, const RouteRule& rule, int* out_id, float* out_gate) {
  if (E <= 128)
    warp_rule_n<4>(zl, E, k, lane, rule, out_id, out_gate);
  else
    warp_rule_n<kMaxEPerLane>(zl, E, k, lane, rule, out_id, out_gate);
}

// A token's logits from memory, a row of E: this lane's.
__device__ __forceinline__ void load_logits(const float* z, int E, int lane, float (&zl)[kMaxEPerLane]) {
#pragma unroll
  for (int m = 0; m < kMaxEPerLane; ++m) {
    const int e = lane + 32 * m;
    zl[m] = e < E ? __ldcg(z + e) : -INFINITY;
  }
}

// The counterparts of route_in_smem and route_one_in_smem under a rule; the gates are made with the choice.
template <int NT>
__device__ void route_in_smem_by_rule(const float* logits, int T, int E, int k, int S, const RouteRule& rule, SmemRouting& r) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < E + S; i += NT) r.mask[i] = 0;
  __syncthreads();
  for (int t = warp; t < T; t += NT / 32) {
    float zl[kMaxEPerLane], gate;
    int id;
    load_logits(logits + t * E, E, lane, zl);
    warp_rule(zl, E, k, lane, rule, &id, &gate);
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
    float zl[kMaxEPerLane], gate;
    int id;
    load_logits(logits, E, lane, zl);
    warp_rule(zl, E, k, lane, rule, &id, &gate);
    if (lane < k) r.gates[lane] = gate;
    if (S && lane == 0) r.gates[k] = 1.0f;
    group_one_in_smem(id, E, k, S, r, lane);
  }
  __syncthreads();
}

}  // namespace dev
}  // namespace fw
