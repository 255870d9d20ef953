// Quantisation to 8-bit blocks: activations (128 neighbours of a token) and
// weights (128 x 128).
#include <algorithm>

#include "fp8.cuh"

namespace fw {
namespace {

using namespace dev;

// Activations: 16 lanes a block, eight values a lane; a warp takes kPairs pairs of
// neighbouring blocks of a token at once, all loads in flight, and a CTA's warps eight
// neighbouring tokens, whose scales lie side by side. Bound by HBM: 2 bytes in, 1 out.
// (Blocks numbered through, a 64-bit division for each found its token: 35 us at 4096 x
// 7168.)
constexpr int kTokens = 8, kPairs = 4;

__global__ void __launch_bounds__(kTokens * 32) fp8_quantize_kernel(const __nv_bfloat16* __restrict__ x, int64_t x_stride, int T, int K, int KB,
                                                                    uint8_t* __restrict__ codes, float* __restrict__ scales, int64_t scale_stride) {
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x * kTokens + (threadIdx.x >> 5);
  if (t >= T) return;
  const __nv_bfloat16* row = x + t * x_stride;
  for (int b0 = blockIdx.y * (2 * kPairs); b0 < KB; b0 += gridDim.y * (2 * kPairs)) {
    uint4 v[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int k = (b0 + 2 * i + half) * kFp8Block + 8 * l;
      v[i] = k < K ? ld_nc_v4(row + k) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int b = b0 + 2 * i + half, k = b * kFp8Block + 8 * l;
      float scale;
      const uint2 c = fp8_block_of_lanes(v[i], &scale);
      if (k < K) *reinterpret_cast<uint2*>(codes + (int64_t)t * K + k) = c;
      if (l == 0 && b < KB) scales[b * scale_stride + t] = scale;
    }
  }
}

// Weights: a CTA a block, a warp taking every eighth row, four values a lane.
// (Done once for each matrix.)
template <bool kFp32>
__global__ void __launch_bounds__(256) fp8_quantize_weight_kernel(const void* __restrict__ w, int N, int K, int KB, uint8_t* __restrict__ codes,
                                                                  float* __restrict__ scales) {
  constexpr int kRows = kFp8Block / 8;
  __shared__ uint32_t s_max[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t block = blockIdx.x;
  const int nb = (int)(block / KB), kb = (int)(block - (int64_t)nb * KB);
  const int k = kb * kFp8Block + 4 * lane;
  float v[kRows][4];
  uint32_t m = 0;
  pdl_wait();
  pdl_launch_dependents();
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int n = nb * kFp8Block + i * 8 + warp;
    if (n < N && k < K) {
      const int64_t at = (int64_t)n * K + k;
      if constexpr (kFp32) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + at));
        v[i][0] = f.x;
        v[i][1] = f.y;
        v[i][2] = f.z;
        v[i][3] = f.w;
      } else {
        const uint2 f = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + at));
        bf16x2_to_f32(f.x, v[i][0], v[i][1]);
        bf16x2_to_f32(f.y, v[i][2], v[i][3]);
      }
    } else {
      v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) m = ::max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = ::max(m, s_max[i]);
  const float top = __uint_as_float(::max(m, kFp8LeastBits)), r = __fdiv_rn(kFp8Max, top);
  if (threadIdx.x == 0) scales[block] = __fdiv_rn(top, kFp8Max);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int n = nb * kFp8Block + i * 8 + warp;
    if (n < N && k < K)
      *reinterpret_cast<uint32_t*>(codes + (int64_t)n * K + k) = e4m3x2(v[i][0] * r, v[i][1] * r) | e4m3x2(v[i][2] * r, v[i][3] * r) << 16;
  }
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

cudaError_t configure_fp8_quantize() {
  // with the linear kernels' carve-out of shared memory they can start beside it
  return cudaFuncSetAttribute(fp8_quantize_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared);
}

cudaError_t launch_fp8_quantize(const void* x, int64_t x_stride, int T, int K, void* codes, float* scales, int64_t scale_stride, cudaStream_t s) {
  const int KB = fp8_blocks(K), parts = (KB + 2 * kPairs - 1) / (2 * kPairs);
  return launch_dependent(fp8_quantize_kernel, dim3((unsigned)((T - 1) / kTokens + 1), (unsigned)std::min(parts, 65535)), dim3(kTokens * 32), 0, s,
                          static_cast<const __nv_bfloat16*>(x), x_stride, T, K, KB, static_cast<uint8_t*>(codes), scales, scale_stride);
}

}  // namespace fw

using namespace fw;

extern "C" fw_status fw_fp8_quantize(const void* x, int64_t x_stride, int32_t T, int32_t K, void* codes, float* scales, int64_t scale_stride,
                                     void* stream) {
  if (T < 0 || K < 16 || K % 16) return set_error(FW_EINVAL, "fw_fp8_quantize: need T >= 0 and K a positive multiple of 16");
  if (T == 0) return FW_OK;
  if (!x || !codes || !scales) return set_error(FW_EINVAL, "fw_fp8_quantize: null pointer");
  if (x_stride < K || x_stride % 8) return set_error(FW_EINVAL, "fw_fp8_quantize: x_stride must cover K and be a multiple of 8 elements");
  if (scale_stride < T || scale_stride % 4) return set_error(FW_EINVAL, "fw_fp8_quantize: scale_stride must cover T and be a multiple of 4 elements");
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16))
    return set_error(FW_EINVAL, "fw_fp8_quantize: x, codes and scales need 16-byte alignment");
  if (fw_status st = check_device("fw_fp8_quantize: needs an sm_103 device"); st != FW_OK) return st;
  const cudaError_t e = launch_fp8_quantize(x, x_stride, T, K, codes, scales, scale_stride, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_cuda_error(e, "fw_fp8_quantize: launch");
  return FW_OK;
}

extern "C" fw_status fw_fp8_quantize_weight(const void* w, int32_t w_fp32, int32_t N, int32_t K, void* codes, float* scales, void* stream) {
  if (N < 1 || K < 16 || K % 16) return set_error(FW_EINVAL, "fw_fp8_quantize_weight: need N >= 1 and K a positive multiple of 16");
  if (w_fp32 != 0 && w_fp32 != 1) return set_error(FW_EINVAL, "fw_fp8_quantize_weight: w_fp32 must be 0 or 1");
  if (!w || !codes || !scales) return set_error(FW_EINVAL, "fw_fp8_quantize_weight: null pointer");
  if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 4))
    return set_error(FW_EINVAL, "fw_fp8_quantize_weight: w and codes need 16-byte, scales 4-byte alignment");
  if (fw_status st = check_device("fw_fp8_quantize_weight: needs an sm_103 device"); st != FW_OK) return st;
  const int KB = fp8_blocks(K);
  const int64_t ctas = (int64_t)fp8_blocks(N) * KB;
  if (ctas > 0x7FFFFFFF) return set_error(FW_EINVAL, "fw_fp8_quantize_weight: too many blocks for one launch");
  const cudaError_t e = dev::launch_dependent(w_fp32 ? fp8_quantize_weight_kernel<true> : fp8_quantize_weight_kernel<false>, dim3((unsigned)ctas), dim3(256),
                                              0, static_cast<cudaStream_t>(stream), w, N, K, KB, static_cast<uint8_t*>(codes), scales);
  if (e != cudaSuccess) return set_cuda_error(e, "fw_fp8_quantize_weight: launch");
  return FW_OK;
}
