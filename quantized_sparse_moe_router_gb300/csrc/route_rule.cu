// Many tokens under a routing rule: the logits as sums over parts of H, then the
// choice from them with the per-tile expert counts that the grouping goes on from.
#include <algorithm>
#include <type_traits>

#include "fp8.cuh"
#include "pair.cuh"
#include "route_rule.cuh"
#include "tcgen05.cuh"

namespace fw {
namespace {

using namespace dev;

// z = x W_r^T by three bf16 planes whose sum is W_r exactly, smallest first into one
// accumulator (every product is exact). Two CTAs of a cluster take 256 tokens and all
// experts with one instruction, each holding half of the tokens and half of the planes'
// rows, and gridDim.y such pairs share H. Bound by the tensor cores, three times x W_r^T:
// 45 GFLOP at 4096 x 7168 x 256 experts, and there by the 64 KB that an SM takes in for
// each 1536 cycles of them. (128 tokens and 128 experts at a time by single CTAs, which
// read x twice and the planes for half as many tokens: 51 us; this: 31.5.)
constexpr int kPairTok = 128, kPairK = 64;       // tokens of a CTA; a stage's part of H, rows of 128 bytes
constexpr int kPairThreads = 256;                // warp 0: tokens; 1: products; 2: planes; 4-7: results
constexpr int kPairMaxStages = 8;
constexpr uint32_t kPairXBytes = kPairTok * 128;
constexpr uint32_t kPairRing = 226 * 1024 - 2048;

struct PairArgs {
  int T, H, E;
  int rows;    // of a plane in a CTA: half the experts, a multiple of 16
  int stages;
  Meta* meta;
};

__device__ __forceinline__ void mma_pair_bf16(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kSw128DescHi)
      : "memory");
}

__global__ void __launch_bounds__(kPairThreads, 1) route_logits_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                                                                       const __grid_constant__ CUtensorMap map_z, const PairArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kPairMaxStages], empty[kPairMaxStages], acc_full;
  __shared__ uint32_t s_tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1, t0 = blockIdx.x * kPairTok;
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // [stages][tokens 128 x 128, 3 planes rows x 128]
  const uint32_t plane = a.rows * 128u, stage = kPairXBytes + 3 * plane;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&acc_full, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(256) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are set up, and their tensor memory is there
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int steps_all = a.H / kPairK, first = (int)((int64_t)steps_all * blockIdx.y / gridDim.y);
  const int steps = (int)((int64_t)steps_all * (blockIdx.y + 1) / gridDim.y) - first;
  bool ok = true;
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0 || warp == 2) {
    const uint32_t first_full = in_cta(full);
    int i = 0, s = 0;
    uint32_t phase = 1;
    for (; i < steps; ++i) {
      if (!(ok = __all_sync(0xFFFFFFFFu, wait_inline(&empty[s], phase)))) {
        if (lane == 0) report_wait(a.meta, kSiteGemm, i, 0);
        break;
      }
      if (elect_one()) {
        uint8_t* st = ring + s * stage;
        const uint32_t bar = first_full + s * 8;
        if (warp == 0) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * stage);
          tma_pair(st, &map_x, (first + i) * kPairK, t0, bar);
        } else {
          for (int p = 0; p < 3; ++p) tma_pair(st + kPairXBytes + p * plane, &map_w, (first + i) * kPairK, p * a.E + rank * a.rows, bar);
        }
      }
      __syncwarp();
      if (++s == a.stages) s = 0, phase ^= 1;
    }
    // (after a wait that gave up) both CTAs' copies in flight land before either leaves
    if (!ok && rank == 0 && warp == 0)
      for (int j = ::max(0, i - a.stages); j < i; ++j) wait_inline(&full[j % a.stages], (j / a.stages) & 1);
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t ring_lo = __shfl_sync(0xFFFFFFFFu, sw128_desc_lo(smem_u32(ring)), 0), acc = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint32_t idesc = idesc_bf16(2 * kPairTok, 2 * a.rows);
      int s = 0;
      uint32_t phase = 0;
      for (int i = 0; i < steps; ++i) {
        if (!__all_sync(0xFFFFFFFFu, wait_inline(&full[s], phase))) {
          if (lane == 0) report_wait(a.meta, kSiteGemm, i, 1);
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t x = ring_lo + s * (stage >> 4), w = x + (kPairXBytes >> 4);
#pragma unroll
          for (int k = 0; k < kPairK / 16; ++k)
#pragma unroll
            for (int p = 2; p >= 0; --p) mma_pair_bf16(acc, x + 2 * k, w + p * (plane >> 4) + 2 * k, idesc, (i | k | (2 - p)) != 0);
          commit_pair(&empty[s]);
        }
        __syncwarp();
        if (++s == a.stages) s = 0, phase ^= 1;
      }
      if (elect_one()) commit_pair(&acc_full);  // (whatever was issued)
      __syncwarp();
      wait_inline(&acc_full, 0);                // no product outlives the tensor memory
    }
  } else if (warp >= 4) {
    const int q = warp & 3, row0 = t0 + 32 * q, chunks = (a.E + 31) / 32;
    if (!__all_sync(0xFFFFFFFFu, wait_inline(&acc_full, 0))) {
      if (lane == 0) report_wait(a.meta, kSiteGemm, 0, 2);
    } else {
      // The ring is free now: 32 tokens by 32 experts at a time, the 16-byte chunk j of a row at j ^ (row % 8)
      tc_fence_after();
      for (int c = 0; c < chunks; ++c) {
        uint32_t v[32];
        tmem_ld(tmem + ((uint32_t)(32 * q) << 16) + 32 * c, v);
        uint8_t* at = ring + (q * chunks + c) * 4096;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(at + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < a.T) tma_out(&map_z, at, 32 * c, row0, blockIdx.y);
      }
      if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves, or gives its tensor memory back, while the other's products or signals reach it
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256) : "memory");
}

// A warp a token, kRouteTileM tokens a CTA (the tiles of the counts). Bound by its
// instructions, some 1300 a token, and the loads before them: a lane's eight logits of
// a part come with one load, four parts in flight (with 4-byte loads a part at a time,
// and the groups over the whole warp, 4096 tokens of 256 experts in 4 parts took 6 us more).
// (1024 threads leave 64 registers each; 76 bytes go to local memory.)
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
    // the parts in order, four parts' loads in flight; then the bias
    const auto load = [&](auto& z) {
      constexpr int kMine = std::extent_v<std::remove_reference_t<decltype(z)>>;
#pragma unroll
      for (int j = 0; j < kMine; ++j) z[j] = 0.f;
      for (int q0 = 0; q0 < parts; q0 += 4) {
        float v[4][kMine];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q0 + q < parts) load_mine(zpart + ((size_t)(q0 + q) * T + t) * E, lane, E, -INFINITY, v[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < kMine; ++j)
            if (q0 + q < parts) z[j] += v[q][j];
      }
      if (zbias) {
        float v[kMine];
        load_mine(zbias, lane, E, 0.f, v);
#pragma unroll
        for (int j = 0; j < kMine; ++j) z[j] += v[j];
      }
    };
    int id;
    float gate;
    warp_rule(load, E, k, lane, rule, &id, &gate);
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

cudaError_t configure_route_rule_kernels() {
  cudaError_t e = configure_tensor_maps();
  if (e == cudaSuccess) e = cudaFuncSetAttribute(route_logits_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairRing + 1024);
  return e;
}

cudaError_t launch_route_rule_logits(Handle* h, const __nv_bfloat16* x, int T, int* parts, cudaStream_t s) {
  const int H = h->cfg.H, E = h->cfg.E, steps = H / kPairK, pairs = h->num_sms / 2, tiles = (T + 2 * kPairTok - 1) / (2 * kPairTok);
  // H is split for the least time, in fifths of a step (0.8 us): a pair's steps, 8 more for
  // starting and ending, and three fifths for a part that the choice then reads (16 tokens
  // of 7168: in 8 parts 27.4 us, in 16 24.5; of 4096: 22.5 and 23.0)
  int n = 1;
  int64_t least = INT64_MAX;
  for (int c = 1; c <= std::min(T <= kRuleSplitT ? kRuleMaxSplit : kRouterMaxSplit, steps); ++c) {
    const int64_t cost = (((int64_t)tiles * c + pairs - 1) / pairs) * ((steps + c - 1) / c + 8) * 5 + 3 * c;
    if (cost < least) least = cost, n = c;
  }
  PairArgs a;
  a.T = T;
  a.H = H;
  a.E = E;
  a.rows = (E + 31) / 32 * 16;
  const uint32_t stage = kPairXBytes + 3 * a.rows * 128;
  a.stages = (int)std::min<uint32_t>(kPairMaxStages, kPairRing / stage);
  a.meta = h->meta;
  CUtensorMap map_x, map_w, map_z;
  cudaError_t e = encode_rows(&map_x, x, false, T, H, (int64_t)H * 2, kPairTok);
  if (e == cudaSuccess) e = encode_rows(&map_w, h->wr3, false, 3 * (int64_t)E, H, (int64_t)H * 2, a.rows);
  if (e == cudaSuccess) e = encode_parts(&map_z, h->zpart, n, T, E, 32);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * tiles), (unsigned)n);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = a.stages * stage + 1024;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  *parts = n;
  return cudaLaunchKernelEx(&cfg, route_logits_kernel, map_x, map_w, map_z, a);
}

cudaError_t launch_route_rule_select(Handle* h, int T, int parts, const float* zbias, int32_t* ids_out, float* gates_out, cudaStream_t s) {
  return launch_dependent(route_rule_select_kernel, dim3((unsigned)((T + kRouteTileM - 1) / kRouteTileM)), dim3(kRouteTileM * 32), 0, s,
                          (const float*)h->zpart, parts, zbias, T, (int)h->cfg.E, (int)h->cfg.k, h->rule, h->ids, h->gates, ids_out, gates_out, h->hist);
}

}  // namespace fw
