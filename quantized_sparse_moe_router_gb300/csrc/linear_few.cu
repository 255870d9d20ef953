// Linear layers in 8 bits for few tokens: the weights are read once and bound
// the call, by HBM.
//
//   out[t][n] = sum_b xs[b][t] ws[n / 128][b] (sum_{k in block b} xc[t][k] wc[n][k])
//
// The weights are the tensor core's A operand: a tile is 128 outputs by one
// block of 128 along K, so it has one scale; the tokens are B (kTok columns).
// The inner sum over a block is made in tensor memory; four warps read it,
// scale it and add it to sums in registers while the next block's runs -- the
// scales are any fp32 numbers, which the tensor core cannot apply.
//
// A cluster of up to eight CTAs shares one tile of 128 outputs, each with a part
// of K: two CTAs on every SM stream weights at once whatever N is. Their sums
// are added in the order of their ranks through distributed shared memory, so
// results do not depend on timing.
//
// Warps: 0 copies (weights, and the tokens' codes), 1 issues the products, 2-5
// scale and add (one tensor-memory quarter each), then either four that
// quantise bf16 tokens straight into the stage (at most 16 tokens: a launch and
// a trip through memory less) or one that fetches scales.
#include <cudaTypedefs.h>

#include <algorithm>

#include "fp8.cuh"
#include "tcgen05.cuh"

namespace fw {
namespace {

using namespace dev;

constexpr int kRows = 128;                           // outputs of a tile: the height of a weight block
constexpr uint32_t kWBytes = kRows * kFp8Block;
constexpr int kLastWarp = 6;                         // warps 2-5 scale and add; from 6 on: quantisers, or the fetcher of scales
constexpr int kMaxCluster = 8;
constexpr uint32_t kSmemHalf = 113 * 1024;           // for two CTAs on an SM

template <int kTok>
struct Few {
  static constexpr uint32_t XBytes = kTok * kFp8Block, StageBytes = kWBytes + XBytes;
  static constexpr int Stages = (int)((kSmemHalf - 1024 - 512) / (StageBytes + kTok * 4));
  static constexpr int Acc = kTok <= 32 ? 4 : 2;     // buffers of sums in tensor memory
  static constexpr uint32_t Cols = Acc * kTok < 32 ? 32 : Acc * kTok;
  static constexpr uint32_t SmemBytes = 1024 + Stages * (StageBytes + kTok * 4);
  static_assert(Cols <= 256, "two CTAs share tensor memory");
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

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The float at this CTA's shared address `addr`, in the CTA of rank `rank` of the cluster.
__device__ __forceinline__ float ld_peer(uint32_t addr, uint32_t rank) {
  uint32_t at;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void store_out(const LinearArgs& a, int t, int n, float v) {
  const int64_t at = (int64_t)t * a.out_stride + n;
  if (a.out_fp32)
    static_cast<float*>(a.out)[at] = v;
  else
    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}

template <int kTok, bool kQuant>
__global__ void __launch_bounds__((kLastWarp + (kQuant ? 4 : 1)) * 32, 2)
    linear_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const LinearArgs a, const int split) {
  using F = Few<kTok>;
  constexpr int kStages = F::Stages, kAcc = F::Acc;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], acc_full[kAcc], acc_empty[kAcc];
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* ring = smem_raw + pad;                                                    // [kStages][weights 128 x 128, tokens kTok x 128]
  float* s_scale = reinterpret_cast<float*>(ring + kStages * F::StageBytes);         // [kStages][kTok] scales, token's times weights'
  const int rank = blockIdx.x % split, tile = blockIdx.x / split;
  const int n0 = tile * kRows, t0 = blockIdx.y * kTok, nt = ::min(kTok, a.T - t0);
  const int b0 = (int)((int64_t)a.KB * rank / split), b1 = (int)((int64_t)a.KB * (rank + 1) / split);
  const float* ws = a.w_scale + (int64_t)tile * a.KB;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1 + (kQuant ? 4 : 1));  // the copies, and the warps that write scales
      mbar_init(&empty[i], 1 + 4);                // the products, and the warps that have read the scales
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
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
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait(bar, parity)) {
      raise(a.status, FW_KV_TIMEOUT);
      ok = false;
    }
    return ok;
  };
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      int i = 0;
      for (int b = b0; b < b1; ++b, ++i) {
        const int s = i % kStages;
        if (!wait(&empty[s], ((i / kStages) & 1) ^ 1)) break;
        uint8_t* st = ring + s * F::StageBytes;
        mbar_arrive_expect_tx(&full[s], kWBytes + (kQuant ? 0u : F::XBytes));
        tma_2d(st, &map_w, b * kFp8Block, n0, &full[s]);
        if (!kQuant) tma_2d(st + kWBytes, &map_x, b * kFp8Block, t0, &full[s]);
      }
      // copies still in flight after a wait that gave up land before the CTA leaves
      if (!ok)
        for (int j = ::max(0, i - kStages); j < i; ++j) mbar_wait(&full[j % kStages], (j / kStages) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int i = 0;
      for (int b = b0; b < b1; ++b, ++i) {
        const int s = i % kStages, c = i % kAcc;
        if (!wait(&full[s], (i / kStages) & 1) || !wait(&acc_empty[c], ((i / kAcc) & 1) ^ 1)) break;
        tc_fence_after();
        const uint32_t w = sw128_desc_lo(smem_u32(ring + s * F::StageBytes)), x = sw128_desc_lo(smem_u32(ring + s * F::StageBytes + kWBytes));
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f8(tmem + c * kTok, w + 2 * k, x + 2 * k, idesc_e4m3(kRows, kTok), k != 0);
        mma_commit(&empty[s]);
        mma_commit(&acc_full[c]);
      }
      if (i > 0) mbar_wait(&acc_full[(i - 1) % kAcc], ((i - 1) / kAcc) & 1);  // no product outlives the tensor memory
    }
  } else if (warp < kLastWarp) {
    const int q = warp & 3;
    float acc[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j) acc[j] = 0.f;
    int i = 0;
    for (int b = b0; b < b1; ++b, ++i) {
      const int s = i % kStages, c = i % kAcc;
      // (the stage's scales are there since before its products began)
      bool fine = mbar_wait(&full[s], (i / kStages) & 1) && mbar_wait(&acc_full[c], (i / kAcc) & 1);
      if (!__all_sync(0xFFFFFFFFu, fine)) {
        raise(a.status, FW_KV_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint32_t from = tmem + ((uint32_t)(32 * q) << 16) + c * kTok;
      const float4* sc = reinterpret_cast<const float4*>(s_scale + s * kTok);
#pragma unroll
      for (int j0 = 0; j0 < kTok; j0 += 16) {
        uint32_t v[16];
        tmem_load(from + j0, v);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = sc[(j0 + j) / 4];
          acc[j0 + j] = fmaf(__uint_as_float(v[j]), f.x, acc[j0 + j]);
          acc[j0 + j + 1] = fmaf(__uint_as_float(v[j + 1]), f.y, acc[j0 + j + 1]);
          acc[j0 + j + 2] = fmaf(__uint_as_float(v[j + 2]), f.z, acc[j0 + j + 2]);
          acc[j0 + j + 3] = fmaf(__uint_as_float(v[j + 3]), f.w, acc[j0 + j + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&acc_empty[c]);
        mbar_arrive(&empty[s]);
      }
    }
    const int row = 32 * q + lane;
    if (split == 1) {
      if (n0 + row < a.N) {
#pragma unroll
        for (int j = 0; j < kTok; ++j)
          if (j < nt) store_out(a, t0 + j, n0 + row, acc[j]);
      }
    } else {  // (every copy has landed and every product has read it: the last block's sums are complete)
      float* part = reinterpret_cast<float*>(ring);  // [kTok][128]
#pragma unroll
      for (int j = 0; j < kTok; ++j) part[j * kRows + row] = acc[j];
    }
  } else if constexpr (kQuant) {
    // 128 threads: rows r and r + 8 of the block, eight values each; the next block's values are fetched ahead
    const int r = (tid - kLastWarp * 32) >> 4, ch = tid & 15;
    auto fetch = [&](int b, uint4 (&v)[2]) {
      const int k = b * kFp8Block + 8 * ch;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = r + 8 * h;
        v[h] = t < nt && k < a.K && b < b1 ? ld_nc_v4(a.x + (int64_t)(t0 + t) * a.x_stride + k) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    uint4 now[2], next[2];
    fetch(b0, now);
    int i = 0;
    for (int b = b0; b < b1; ++b, ++i) {
      const int s = i % kStages;
      fetch(b + 1, next);
      const float w = __ldg(ws + b);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[s], ((i / kStages) & 1) ^ 1))) {
        raise(a.status, FW_KV_TIMEOUT);
        break;
      }
      uint8_t* x = ring + s * F::StageBytes + kWBytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (8 * h < nt || h == 0) {
          const int t = r + 8 * h;
          float scale;
          const uint2 c = fp8_block_of_lanes(now[h], &scale);
          // (chunk of 16 bytes j of row t lies at j ^ (t % 8): the 128-byte swizzle)
          *reinterpret_cast<uint2*>(x + t * kFp8Block + (((ch >> 1) ^ (t & 7)) << 4) + 8 * (ch & 1)) = c;
          if (ch == 0) s_scale[s * kTok + t] = scale * w;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
      now[0] = next[0];
      now[1] = next[1];
    }
  } else {
    // one warp: the tokens' scales times the weights', a block ahead
    constexpr int kPer = (kTok + 31) / 32;
    auto fetch = [&](int b, float (&v)[kPer]) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int t = lane + 32 * j;
        v[j] = t < nt && b < b1 ? __ldg(a.x_scale + (int64_t)b * a.T + t0 + t) * __ldg(ws + b) : 0.f;
      }
    };
    float now[kPer], next[kPer];
    fetch(b0, now);
    int i = 0;
    for (int b = b0; b < b1; ++b, ++i) {
      const int s = i % kStages;
      fetch(b + 1, next);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[s], ((i / kStages) & 1) ^ 1))) {
        raise(a.status, FW_KV_TIMEOUT);
        break;
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (lane + 32 * j < kTok) s_scale[s * kTok + lane + 32 * j] = now[j];
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
#pragma unroll
      for (int j = 0; j < kPer; ++j) now[j] = next[j];
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F::Cols) : "memory");
  if (split > 1) {
    cluster_sync();  // every CTA's sums are in its shared memory
    const int all = nt * kRows, i0 = all * rank / split, i1 = all * (rank + 1) / split;
    const uint32_t part = smem_u32(ring);
    for (int i = i0 + tid; i < i1; i += (int)blockDim.x) {
      const int n = n0 + i % kRows;
      float v = 0.f;
      for (int r = 0; r < split; ++r) v += ld_peer(part + 4 * i, r);
      if (n < a.N) store_out(a, t0 + i / kRows, n, v);
    }
    cluster_sync();  // none leaves while another still reads its sums
  }
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

template <int kTok, bool kQuant>
cudaError_t configure() {
  cudaError_t e = cudaFuncSetAttribute(linear_few_kernel<kTok, kQuant>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Few<kTok>::SmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(linear_few_kernel<kTok, kQuant>, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared);
  return e;
}

template <int kTok, bool kQuant>
cudaError_t launch(const LinearArgs& a, const void* w, const void* x_codes, int64_t codes_stride, int sms, cudaStream_t s) {
  CUtensorMap map_w, map_x = {};
  cudaError_t e = encode_codes(&map_w, w, a.N, a.K, a.K, kRows);
  if (e == cudaSuccess && !kQuant) e = encode_codes(&map_x, x_codes, a.T, a.K, codes_stride, kTok);
  if (e != cudaSuccess) return e;
  // parts of K: as many as still find room beside each other, two CTAs an SM, with two blocks each at least
  const int64_t tiles = (int64_t)((a.N + kRows - 1) / kRows) * ((a.T + kTok - 1) / kTok);
  int split = 1;
  while (split < kMaxCluster && tiles * split * 2 <= 2 * sms && a.KB >= split * 4) split *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + kRows - 1) / kRows * split), (unsigned)((a.T + kTok - 1) / kTok));
  cfg.blockDim = dim3((kLastWarp + (kQuant ? 4 : 1)) * 32);
  cfg.dynamicSmemBytes = Few<kTok>::SmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_few_kernel<kTok, kQuant>, map_w, map_x, a, split);
}

}  // namespace

cudaError_t encode_codes(CUtensorMap* map, const void* codes, int64_t rows, int64_t K, int64_t stride, int box) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
  const cuuint32_t boxes[2] = {(cuuint32_t)kFp8Block, (cuuint32_t)box}, steps[2] = {1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

bool linear_few_quantises(int T) { return T <= 16; }

cudaError_t configure_linear_few() {
  if (!g_encode) {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  cudaError_t e = configure<16, true>();
  if (e == cudaSuccess) e = configure<16, false>();
  if (e == cudaSuccess) e = configure<32, false>();
  if (e == cudaSuccess) e = configure<64, false>();
  if (e == cudaSuccess) e = configure<128, false>();
  return e;
}

cudaError_t launch_linear_few(const LinearArgs& a, const void* w, const void* x_codes, int64_t codes_stride, int sms, cudaStream_t s) {
  if (a.x) return launch<16, true>(a, w, nullptr, 0, sms, s);
  if (a.T <= 16) return launch<16, false>(a, w, x_codes, codes_stride, sms, s);
  if (a.T <= 32) return launch<32, false>(a, w, x_codes, codes_stride, sms, s);
  if (a.T <= 64) return launch<64, false>(a, w, x_codes, codes_stride, sms, s);
  return launch<128, false>(a, w, x_codes, codes_stride, sms, s);
}

}  // namespace fw
