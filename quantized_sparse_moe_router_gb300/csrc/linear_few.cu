// Linear layers in 8 bits for few tokens: the weights are read once and bound
// the call, by HBM.
//
//   out[t][n] = sum_b xs[b][t] ws[n / 128][b] (sum_{k in block b} xc[t][k] wc[n][k])
//
// The weights are the tensor core's A operand: a tile is 128 outputs by one
// block of 128 along K, so it has one scale; the tokens are B (kTok columns).
// The inner sum over a block is made in tensor memory; four or eight warps read it,
// scale it and add it to sums in registers while the next block's runs -- the
// scales are any fp32 numbers, which the tensor core cannot apply.
//
// Where there are fewer tiles of 128 outputs than CTAs find room, a cluster of up to
// eight CTAs shares one, each with a part of K; their sums are added in the order of
// their ranks through distributed shared memory, so results do not depend on timing.
// Where there are more, a CTA takes several tiles, and its copies run on from one to
// the next.
//
// Warps: 0 copies weights, 1 issues the products, 2 copies the tokens' codes and
// scales, 4 on scale and add (tensor-memory quarter = warp % 4). With at most 16
// bf16 tokens it copies those, and four more warps quantise them within the stage (a
// launch and a trip through memory less; loaded by these warps, two blocks ahead, their
// latency bounded them).

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fp8.cuh"
#include "pair.cuh"
#include "tcgen05.cuh"

namespace fw {
namespace {

using namespace dev;

constexpr int kRows = 128;                           // outputs of a tile: the height of a weight block
constexpr uint32_t kWBytes = kRows * kFp8Block;
constexpr int kFirstEpi = 4, kQuantWarps = 4;
constexpr int kMaxCluster = 8;

// kQuant: a stage also holds the tokens as they come, 128 bf16 values each.
template <int kTok, bool kQuant>
struct Few {
  static constexpr int Ctas = kTok <= 64 ? 2 : 1;    // on an SM
  static constexpr int Both = kTok <= 16 ? 120 : Ctas == 2 ? 175 : 200;  // (see split_of)
  static constexpr int EpiWarps = kTok <= 32 ? 4 : 8;
  static constexpr int Mine = kTok * 4 / EpiWarps;   // columns of a scaling thread
  static constexpr int Slot = kTok < 32 ? 32 : kTok; // scales of a stage (copies of them start on 128 bytes)
  static constexpr uint32_t XBytes = kTok * kFp8Block, RawBytes = kQuant ? 2 * XBytes : 0, StageBytes = kWBytes + XBytes + RawBytes, ScaleBytes = Slot * 4;
  static constexpr int Stages = (int)(((Ctas == 2 ? 113 : 226) * 1024 - 1024 - 512) / (StageBytes + ScaleBytes));
  static constexpr int Acc = 4;                      // buffers of sums in tensor memory: the way round one is about 1,200 cycles, the products 480
  static constexpr uint32_t Cols = Acc * kTok;
  // Not less than 110 KB: the fused expert kernel (122 KB or more) lets its dependents start
  // before it takes its tensor memory. Beside it on an SM this one would take some first, and
  // hold it until that kernel's end, for which it waits; so there must be no room beside it.
  static constexpr uint32_t LeastSmem = 110 * 1024, UsedSmem = 1024 + Stages * (StageBytes + ScaleBytes);
  static constexpr uint32_t SmemBytes = UsedSmem < LeastSmem ? LeastSmem : UsedSmem;
  static_assert(Cols >= 32 && Cols * Ctas <= 512 && (Cols & (Cols - 1)) == 0, "an SM's CTAs share tensor memory");
  static_assert(kRows * kTok * 4 <= Stages * StageBytes, "the partial sums take the ring's place");
};

// kind::f8f6f4, D fp32, A and B e4m3, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kSw128DescHi)
      : "memory");
}

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// acc += v f w (kJoined: see scales_join).
template <bool kJoined>
__device__ __forceinline__ void add_scaled(float& acc, uint32_t v, float f, float w) {
  acc = kJoined ? fmaf(__uint_as_float(v), f * w, acc) : fmaf(__uint_as_float(v) * w, f, acc);
}

__device__ __forceinline__ void store_out(const LinearArgs& a, int t, int n, float v) {
  const int64_t at = (int64_t)t * a.out_stride + n;
  if (a.out_fp32)
    static_cast<float*>(a.out)[at] = v;
  else
    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}

// Four neighbouring outputs of a token, n a multiple of four.
__device__ __forceinline__ void store_four(const LinearArgs& a, int t, int n, float4 v) {
  const int64_t at = (int64_t)t * a.out_stride + n;
  const uintptr_t to = reinterpret_cast<uintptr_t>(a.out) + at * (a.out_fp32 ? 4 : 2);
  if (n + 4 <= a.N && to % (a.out_fp32 ? 16 : 8) == 0) {
    if (a.out_fp32)
      *reinterpret_cast<float4*>(to) = v;
    else
      *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2_bits(v.x, v.y), bf16x2_bits(v.z, v.w));
    return;
  }
  if (n < a.N) store_out(a, t, n, v.x);
  if (n + 1 < a.N) store_out(a, t, n + 1, v.y);
  if (n + 2 < a.N) store_out(a, t, n + 2, v.z);
  if (n + 3 < a.N) store_out(a, t, n + 3, v.w);
}

template <int kTok, bool kQuant>
constexpr int few_threads() {
  return (kFirstEpi + Few<kTok, kQuant>::EpiWarps + (kQuant ? kQuantWarps : 0)) * 32;
}

// tiles: of 128 outputs; split: CTAs that share one (more than one: a CTA has one tile).
template <int kTok, bool kQuant>
__global__ void __launch_bounds__(few_threads<kTok, kQuant>(), Few<kTok, kQuant>::Ctas)
    linear_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_s,
                      const LinearArgs a, const int tiles, const int split) {
  using F = Few<kTok, kQuant>;
  constexpr int kStages = F::Stages, kAcc = F::Acc, kMine = F::Mine;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], raw_full[kStages], acc_full[kAcc], acc_empty[kAcc];
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* ring = smem_raw + pad;                                                    // [kStages][weights 128 x 128, tokens kTok x 128, raw]
  float* s_scale = reinterpret_cast<float*>(ring + kStages * F::StageBytes);         // [kStages][Slot] the tokens' scales
  const int rank = blockIdx.x % split, first = blockIdx.x / split, step = gridDim.x / split;
  const int t0 = blockIdx.y * kTok, nt = ::min(kTok, a.T - t0);
  const int b0 = (int)((int64_t)a.KB * rank / split), nb = (int)((int64_t)a.KB * (rank + 1) / split) - b0;  // this CTA's blocks of K
  const int blocks = first < tiles ? ((tiles - first + step - 1) / step) * nb : 0;                          // over all its tiles

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1 + (kQuant ? kQuantWarps : 1));  // the weights' copies; the tokens'
      mbar_init(&raw_full[i], 1);
      mbar_init(&empty[i], 1 + F::EpiWarps);                // the products, and the warps that have read the scales
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], F::EpiWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(F::Cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // by a whole warp, which stays together
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = __all_sync(0xFFFFFFFFu, wait_inline(bar, parity));
    if (!ok) raise(a.status, FW_KV_TIMEOUT);
    return ok;
  };
  if (!a.x_alone || warp == 2) pdl_wait();
  pdl_launch_dependents();

  if (warp == 0 || warp == 2) {
    bool ok = true;
    int i = 0, s = 0, b = 0, tile = first;
    uint32_t phase = 1;
    for (; i < blocks; ++i) {
      if (!(ok = wait(&empty[s], phase))) break;
      if (elect_one()) {
        uint8_t* st = ring + s * F::StageBytes;
        if (warp == 0) {
          mbar_arrive_expect_tx(&full[s], kWBytes);
          tma_2d(st, &map_w, (b0 + b) * kFp8Block, tile * kRows, &full[s]);
        } else if constexpr (kQuant) {
          mbar_arrive_expect_tx(&raw_full[s], F::RawBytes);
          tma_2d(st + kWBytes + F::XBytes, &map_x, (b0 + b) * kFp8Block, t0, &raw_full[s]);
        } else {
          mbar_arrive_expect_tx(&full[s], F::XBytes + F::ScaleBytes);
          tma_2d(st + kWBytes, &map_x, (b0 + b) * kFp8Block, t0, &full[s]);
          tma_2d(s_scale + s * F::Slot, &map_s, t0, b0 + b, &full[s]);
        }
      }
      __syncwarp();
      if (++b == nb) b = 0, tile += step;
      if (++s == kStages) s = 0, phase ^= 1;
    }
    // copies still in flight after a wait that gave up land before the CTA leaves
    if (!ok)
      for (int j = ::max(0, i - kStages); j < i; ++j) wait_inline(kQuant && warp == 2 ? &raw_full[j % kStages] : &full[j % kStages], (j / kStages) & 1);
  } else if (warp == 1) {
    // (descriptors from a value shuffled from lane 0 are uniform for the compiler)
    const uint32_t ring_lo = __shfl_sync(0xFFFFFFFFu, sw128_desc_lo(smem_u32(ring)), 0), cols0 = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    int i = 0, s = 0;
    uint32_t phase = 0;
    for (; i < blocks; ++i) {
      const int c = i % kAcc;
      const uint32_t c_phase = ((i / kAcc) & 1) ^ 1;
      // (both are asked at once: an answer takes some 70 cycles)
      const bool f = mbar_test(&full[s], phase), e = mbar_test(&acc_empty[c], c_phase);
      if (!__all_sync(0xFFFFFFFFu, f && e) && !(wait(&full[s], phase) && wait(&acc_empty[c], c_phase))) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t w = ring_lo + s * (F::StageBytes >> 4), x = w + (kWBytes >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f8(cols0 + c * kTok, w + 2 * k, x + 2 * k, idesc_e4m3(kRows, kTok), k != 0);
        mma_commit(&acc_full[c]);
        mma_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == kStages) s = 0, phase ^= 1;
    }
    if (i > 0) wait_inline(&acc_full[(i - 1) % kAcc], ((i - 1) / kAcc) & 1);  // no product outlives the tensor memory
  } else if (warp >= kFirstEpi && warp < kFirstEpi + F::EpiWarps) {
    const int q = warp & 3, part = (warp - kFirstEpi) >> 2, row = 32 * q + lane;
    const uint32_t from0 = tmem + ((uint32_t)(32 * q) << 16) + part * kMine;
    bool ok = true;
    int i = 0, s = 0;
    uint32_t phase = 0;
    for (int tile = first; tile < tiles && ok; tile += step) {
      const float* ws = a.w_scale + (int64_t)tile * a.KB + b0;
      float w_now = 0.f, w_next = lane < nb ? __ldg(ws + lane) : 0.f;  // the weights' scales of 32 blocks, one a lane
      float acc[kMine];
#pragma unroll
      for (int j = 0; j < kMine; ++j) acc[j] = 0.f;
      const auto add_blocks = [&](auto joined, int b, int end) {
        for (; b < end; ++b, ++i) {
          const float w = __shfl_sync(0xFFFFFFFFu, w_now, b % 32);
          const int c = i % kAcc;
          const uint32_t c_phase = (i / kAcc) & 1;
          // (the stage's scales are there since before its products began)
          const bool f = mbar_test(&full[s], phase), e = mbar_test(&acc_full[c], c_phase);
          if (!__all_sync(0xFFFFFFFFu, f && e) && !(ok = wait(&full[s], phase) && wait(&acc_full[c], c_phase))) break;
          tc_fence_after();
          const uint32_t from = from0 + c * kTok;
          const float4* sc = reinterpret_cast<const float4*>(s_scale + s * F::Slot + part * kMine);
#pragma unroll
          for (int j0 = 0; j0 < kMine; j0 += 16) {
            uint32_t v[16];
            tmem_load(from + j0, v);
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 f = sc[(j0 + j) / 4];
              add_scaled<joined>(acc[j0 + j], v[j], f.x, w);
              add_scaled<joined>(acc[j0 + j + 1], v[j + 1], f.y, w);
              add_scaled<joined>(acc[j0 + j + 2], v[j + 2], f.z, w);
              add_scaled<joined>(acc[j0 + j + 3], v[j + 3], f.w, w);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&acc_empty[c]);
            mbar_arrive(&empty[s]);
          }
          if (++s == kStages) s = 0, phase ^= 1;
        }
      };
      for (int b = 0; b < nb && ok; b += 32) {
        w_now = w_next;
        w_next = b + 32 + lane < nb ? __ldg(ws + b + 32 + lane) : 0.f;
        if (__all_sync(0xFFFFFFFFu, b + lane >= nb || scales_join(w_now)))
          add_blocks(std::true_type(), b, ::min(nb, b + 32));
        else
          add_blocks(std::false_type(), b, ::min(nb, b + 32));
      }
      if (!ok) break;
      if (split == 1) {
        const int n = tile * kRows + row;
        if (n < a.N) {
#pragma unroll
          for (int j = 0; j < kMine; ++j)
            if (part * kMine + j < nt) store_out(a, t0 + part * kMine + j, n, acc[j]);
        }
      } else {  // (every copy has landed and every product has read it: the last block's sums are complete)
        float* sums = reinterpret_cast<float*>(ring);  // [kTok][128]
#pragma unroll
        for (int j = 0; j < kMine; ++j) sums[(part * kMine + j) * kRows + row] = acc[j];
      }
    }
  } else if constexpr (kQuant) {
    if (warp >= kFirstEpi + F::EpiWarps) {
      // 128 threads: rows r, r + 8, .. of a block, eight values each
      const int r = (tid - (kFirstEpi + F::EpiWarps) * 32) >> 4, ch = tid & 15;
      int s = 0;
      uint32_t phase = 0;
      for (int i = 0; i < blocks; ++i) {
        if (!wait(&raw_full[s], phase)) break;
        uint8_t* x = ring + s * F::StageBytes + kWBytes;
#pragma unroll
        for (int h = 0; h < kTok / 8; ++h) {
          if (8 * h < nt) {
            const int t = r + 8 * h;
            float scale;
            const uint2 c = fp8_block_of_lanes(*reinterpret_cast<const uint4*>(x + F::XBytes + t * 256 + ch * 16), &scale);
            // (chunk of 16 bytes j of row t lies at j ^ (t % 8): the 128-byte swizzle)
            *reinterpret_cast<uint2*>(x + t * kFp8Block + (((ch >> 1) ^ (t & 7)) << 4) + 8 * (ch & 1)) = c;
            if (ch == 0) s_scale[s * F::Slot + t] = scale;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        if (++s == kStages) s = 0, phase ^= 1;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F::Cols) : "memory");
  if (split > 1) {
    cluster_sync();  // every CTA's sums are in its shared memory
    // each its share of them, four outputs of a token a thread, all ranks' parts on their way at once
    const int all = nt * (kRows / 4), i0 = all * rank / split, i1 = all * (rank + 1) / split;
    for (int i = i0 + tid; i < i1; i += (int)blockDim.x) {
      float4 p[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) p[r] = r < split ? ld_cta(in_cta(ring + 16 * i, r)) : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 v = p[0];
#pragma unroll
      for (int r = 1; r < kMaxCluster; ++r) v.x += p[r].x, v.y += p[r].y, v.z += p[r].z, v.w += p[r].w;
      store_four(a, t0 + i / (kRows / 4), first * kRows + i % (kRows / 4) * 4, v);
    }
    cluster_sync();  // none leaves while another still reads its sums
  }
}

// Clusters of 2 .. kMaxCluster CTAs that a device runs at once: a cluster's SMs are of one
// group of them, so there are fewer than the SMs have places for.
struct Room {
  std::atomic<int> clusters[kMaxCluster + 1];
  std::atomic<int> alone[kMaxCluster + 1];  // with an SM for each CTA
};
template <int kTok, bool kQuant>
Room& room_of(int dev) {
  static Room room[64];
  return room[dev];
}

template <int kTok, bool kQuant>
cudaError_t configure(int dev) {
  cudaError_t e = cudaFuncSetAttribute(linear_few_kernel<kTok, kQuant>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Few<kTok, kQuant>::SmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(linear_few_kernel<kTok, kQuant>, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared);
  int one[kMaxCluster + 1] = {};  // with an SM for each CTA, which is what is reported
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&one[1], cudaDevAttrMultiProcessorCount, dev);
  for (int c = 2; c <= kMaxCluster && e == cudaSuccess; ++c)
    e = active_clusters(linear_few_kernel<kTok, kQuant>, c, few_threads<kTok, kQuant>(), Few<kTok, kQuant>::SmemBytes, &one[c]);
  // With two CTAs an SM: as many as have half the size; of an odd size, halfway between what
  // is sure (twice as many, or as many as have one CTA more) and what there are places for
  // (96 of three ran at once, 40 of seven did not: 64 x 7168 x 5120 19.0 us, with six of
  // them to a tile 13.1).
  int n = 0;
  for (int c = kMaxCluster; c >= 2; --c) {
    n = Few<kTok, kQuant>::Ctas == 1 ? one[c] : c % 2 ? (std::max(2 * one[c], n) + 2 * one[1] / c) / 2 : one[c / 2];
    room_of<kTok, kQuant>(dev).clusters[c].store(n);
    room_of<kTok, kQuant>(dev).alone[c].store(one[c]);
  }
  return e;
}

// CTAs that share a tile: as many as keep the SM with the most work shortest, in
// blocks of K (*longest), with two for each CTA's beginning and end. All find room at
// once, and a part of K has two blocks at least. Two CTAs on an SM take `both` / 100 of what
// one takes by itself: 120 with up to 16 tokens, whose blocks are mostly latency (16 x 2048 x
// 5120 in 3 parts 7.4 us, in 6 6.7; 16 x 4096 x 4096 in 4 8.9, in 8 7.9), 175 with more
// (64 x 4096 x 2560 in 6 parts 7.0 us, in 8 8.2; 64 x 4096 x 4096 in 4 8.7, in 8 9.8).
int split_of(int tiles, int rows, int KB, const Room& room, int both, int sms, int64_t* longest) {
  const int64_t all = (int64_t)tiles * rows;
  int split = 1;
  int64_t best = (all + sms - 1) / sms * (KB + 2) * (all > sms ? both / 2 : 100);
  for (int c = 2; c <= kMaxCluster && KB >= 2 * c; ++c) {
    if (all > room.clusters[c].load()) continue;
    const int64_t cost = ((KB + c - 1) / c + 2) * (all > room.alone[c].load() ? both : 100);
    if (cost < best) best = cost, split = c;
  }
  if (longest) *longest = best / 100;
  return split;
}

template <int kTok, bool kQuant>
cudaError_t launch(const LinearArgs& a, const void* w, const void* x_codes, int64_t codes_stride, int dev, int sms, cudaStream_t s) {
  CUtensorMap map_w, map_x = {}, map_s = {};
  cudaError_t e = encode_codes(&map_w, w, a.N, a.K, a.K, kRows);
  if (e == cudaSuccess) e = kQuant ? encode_values(&map_x, a.x, a.T, a.K, a.x_stride, kTok) : encode_codes(&map_x, x_codes, a.T, a.K, codes_stride, kTok);
  if (e == cudaSuccess && !kQuant) e = encode_scales(&map_s, a.x_scale, a.T, a.KB, a.x_scale_stride, Few<kTok, kQuant>::Slot);
  if (e != cudaSuccess) return e;
  const int tiles = (a.N + kRows - 1) / kRows, rows = (a.T + kTok - 1) / kTok;
  const int split = split_of(tiles, rows, a.KB, room_of<kTok, kQuant>(dev), Few<kTok, kQuant>::Both, sms, nullptr);
  const int64_t room = (int64_t)Few<kTok, kQuant>::Ctas * sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(split > 1 ? tiles * split : std::min<int64_t>(tiles, std::max<int64_t>(1, room / rows))), (unsigned)rows);
  cfg.blockDim = dim3(few_threads<kTok, kQuant>());
  cfg.dynamicSmemBytes = Few<kTok, kQuant>::SmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_few_kernel<kTok, kQuant>, map_w, map_x, map_s, a, tiles, split);
}

}  // namespace

// (17 to 32 tokens: 12.4 us at 4096 x 4096 against 10.3 with a launch for them)
bool linear_few_quantises(int T) { return T <= 16; }

cudaError_t configure_linear_few(int dev) {
  cudaError_t e = configure_tensor_maps();
  if (e == cudaSuccess) e = configure<16, true>(dev);
  if (e == cudaSuccess) e = configure<16, false>(dev);
  if (e == cudaSuccess) e = configure<32, false>(dev);
  if (e == cudaSuccess) e = configure<64, false>(dev);
  if (e == cudaSuccess) e = configure<128, false>(dev);
  return e;
}

int64_t linear_few_blocks(int T, int N, int KB, int dev, int sms) {
  int64_t longest;
  split_of((N + kRows - 1) / kRows, (T + 127) / 128, KB, room_of<128, false>(dev), Few<128, false>::Both, sms, &longest);
  return longest;
}

cudaError_t launch_linear_few(const LinearArgs& a, const void* w, const void* x_codes, int64_t codes_stride, int dev, int sms, cudaStream_t s) {
  if (a.x) return launch<16, true>(a, w, nullptr, 0, dev, sms, s);
  if (a.T <= 16) return launch<16, false>(a, w, x_codes, codes_stride, dev, sms, s);
  if (a.T <= 32) return launch<32, false>(a, w, x_codes, codes_stride, dev, sms, s);
  if (a.T <= 64) return launch<64, false>(a, w, x_codes, codes_stride, dev, sms, s);
  return launch<128, false>(a, w, x_codes, codes_stride, dev, sms, s);
}

}  // namespace fw
