// Many tokens under a routing rule: the choice from logits that the prefill
// router left as sums over parts of H, and the per-tile expert counts that the
// grouping goes on from.
#include "route_rule.cuh"

namespace fw {
namespace {

using namespace dev;

// A warp a token, kRouteTileM tokens a CTA (the tiles of the counts); latency of
// the warp reductions bounds it, so a token has a warp of its own.
__global__ void __launch_bounds__(kRouteTileM * 32) route_rule_select_kernel(const float* __restrict__ zpart, int parts, const float* __restrict__ zbias, int T,
                                                                             int E, int k, RouteRule rule, int32_t* ids, float* gates, int32_t* ids_out,
                                                                             float* gates_out, int32_t* hist) {
  __shared__ int s_cnt[kMaxE];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x * kRouteTileM + warp;
  for (int i = threadIdx.x; i < E; i += kRouteTileM * 32) s_cnt[i] = 0;
  pdl_wait();  // the partial logits
  pdl_launch_dependents();
  __syncthreads();
  if (t < T) {
    float zl[kMaxEPerLane];
#pragma unroll
    for (int m = 0; m < kMaxEPerLane; ++m) zl[m] = 0.f;
    for (int q = 0; q < parts; ++q) {  // (in order; then the bias)
      const float* zq = zpart + ((size_t)q * T + t) * E;
#pragma unroll
      for (int m = 0; m < kMaxEPerLane; ++m) zl[m] += lane + 32 * m < E ? __ldg(zq + lane + 32 * m) : 0.f;
    }
#pragma unroll
    for (int m = 0; m < kMaxEPerLane; ++m) zl[m] = lane + 32 * m < E ? zl[m] + (zbias ? __ldg(zbias + lane + 32 * m) : 0.f) : -INFINITY;
    int id;
    float gate;
    warp_rule(zl, E, k, lane, rule, &id, &gate);
    if (lane < k) {
      ids[t * k + lane] = id;
      gates[t * k + lane] = gate;
      ids_out[t * k + lane] = id;
      if (gates_out) gates_out[t * k + lane] = gate;
      atomicAdd(&s_cnt[id], 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kRouteTileM * 32) hist[(int64_t)blockIdx.x * E + e] = s_cnt[e];
}

}  // namespace

cudaError_t launch_route_rule_select(Handle* h, int T, int parts, const float* zbias, int32_t* ids_out, float* gates_out, cudaStream_t s) {
  return launch_dependent(route_rule_select_kernel, dim3((unsigned)((T + kRouteTileM - 1) / kRouteTileM)), dim3(kRouteTileM * 32), 0, s,
                          (const float*)h->zpart, parts, zbias, T, (int)h->cfg.E, (int)h->cfg.k, h->rule, h->ids, h->gates, ids_out, gates_out, h->hist);
}

}  // namespace fw
