// Blocks of 8-bit floating point values (e4m3) with a scale, and the linear
// layers over them.
//
//   m = max(largest magnitude, 2^-96),  scale = m / 448,  code = e4m3(x (448 / m))
//
// 448 is e4m3's largest value, so the largest element of a block takes the
// largest code. The least m keeps 448 / m finite (a block of zeros, or of
// subnormals, needs no case of its own: its codes round to zero). The largest
// magnitude of bf16 values is taken on their bits, as whole numbers: an
// infinity is above every number and a NaN above it, so both reach m, and the
// scale takes them into every output of the block.
#pragma once

#include "kvcache.cuh"

namespace fw {

constexpr int kFp8Block = 128;  // values along K that share a scale

__host__ __device__ inline int fp8_blocks(int n) { return n / kFp8Block + (n % kFp8Block != 0); }  // (n + 127 may not fit)

namespace dev {

constexpr uint32_t kFp8LeastBits = 0x0F800000u;  // 2^-96
constexpr float kFp8Max = 448.f;

// The largest magnitude of eight bf16 values, as the bits of a float.
__device__ __forceinline__ uint32_t bf16x8_amax_bits(const uint4 v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  return ::max(m << 16, m & 0xFFFF0000u);
}

// Two fp32 values -> two e4m3 codes (the first in the low byte), nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight bf16 values times r -> eight codes.
__device__ __forceinline__ uint2 bf16x8_to_e4m3(const uint4 v, float r) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    bf16x2_to_f32(w[i], lo, hi);
    c[i] = e4m3x2(lo * r, hi * r);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// A block of 128 bf16 values over 16 neighbouring lanes, eight a lane (all 32
// lanes of the warp take part): this lane's codes, and the block's scale.
__device__ __forceinline__ uint2 fp8_block_of_lanes(const uint4 v, float* scale) {
  uint32_t m = bf16x8_amax_bits(v);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = ::max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float top = __uint_as_float(::max(m, kFp8LeastBits));
  *scale = __fdiv_rn(top, kFp8Max);
  return bf16x8_to_e4m3(v, __fdiv_rn(kFp8Max, top));
}

// Whether the barrier's phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait without a call (around which the caller's registers would have to be
// saved) and without sleep: what waits here is on the way of every block.
__device__ __forceinline__ bool wait_inline(uint64_t* bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i)
    if ((i & 1023u) == 0) {  // (the clock takes long to read)
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) return false;
    }
  return true;
}

// Whether a weight scale's product with a token's is a normal fp32 number whatever the
// token's: those the rule gives lie between 2^-104.9 and 2^119.2. Where it need not be (a
// block of weights all below 2^-12, so also one of zeros, or one above 2^16) a block's sum, 0
// or of 2^-18 to 2^24.6, is multiplied by the weights' scale and then by the token's: what is
// between is above 2^-123, and below 2^128 for weights' scales up to 2^103. Asked for 32
// blocks at a time, with a loop for each way: a branch for each block's additions took 4096 x
// 7168 x 4096 from 91 us to 118, two multiplications for all to 110.
__device__ __forceinline__ bool scales_join(float w) { return fabsf(w) >= 4.76837158203125e-7f && fabsf(w) <= 256.f; }

}  // namespace dev

// What the linear kernels take: codes of the tokens with their scales, or (few
// tokens) bf16 values that the kernel quantises itself.
struct LinearArgs {
  int T, K, N, KB;          // KB = blocks along K
  const __nv_bfloat16* x;   // bf16 [T][x_stride], where the kernel quantises
  int64_t x_stride;
  const float* x_scale;     // [KB] rows of T, x_scale_stride apart
  int64_t x_scale_stride;
  const float* w_scale;     // [ceil(N / 128)][KB]
  void* out;
  int64_t out_stride;
  int out_fp32;
  int32_t* status;
  // The predecessor in the stream is the quantisation of x, which began when all before
  // it was complete: nothing but the tokens' codes and scales has to be waited for.
  int x_alone;
};

cudaError_t configure_fp8_quantize();
cudaError_t launch_fp8_quantize(const void* x, int64_t x_stride, int T, int K, void* codes, float* scales, int64_t scale_stride, cudaStream_t s);

cudaError_t configure_tensor_maps();  // before the first of the encode_* below

// A tensor map of codes: rows of K bytes, `stride` apart, in boxes of 128 bytes by `box` rows, 128-byte swizzle.
cudaError_t encode_codes(CUtensorMap* map, const void* codes, int64_t rows, int64_t K, int64_t stride, int box);

// The same of results (or of bf16 operands): rows of `cols` bf16 or fp32 values, in boxes of 128 bytes by `box` rows, 128-byte swizzle.
cudaError_t encode_rows(CUtensorMap* map, const void* out, bool fp32, int64_t rows, int64_t cols, int64_t row_bytes, int box);

// The same of bf16 values: rows of K, `stride` elements apart, in boxes of 128 by `box` rows, no swizzle.
cudaError_t encode_values(CUtensorMap* map, const __nv_bfloat16* x, int64_t T, int64_t K, int64_t stride, int box);

// The same of tokens' scales: KB rows of T, in boxes of `box` by one row, no swizzle.
cudaError_t encode_scales(CUtensorMap* map, const float* scales, int64_t T, int KB, int64_t stride, int box);

// The same of n fp32 matrices [T][cols], one behind the other, in boxes of 32 columns by `box` rows, 128-byte swizzle.
cudaError_t encode_parts(CUtensorMap* map, float* parts, int n, int64_t T, int64_t cols, int box);

// (dev: the current device, below 64)
cudaError_t configure_linear_few(int dev);
bool linear_few_quantises(int T);  // whether the kernel for few tokens takes bf16 itself
// Blocks of K that an SM takes one after the other at most, at more than 64 tokens.
int64_t linear_few_blocks(int T, int N, int KB, int dev, int sms);
cudaError_t launch_linear_few(const LinearArgs& a, const void* w, const void* x_codes, int64_t codes_stride, int dev, int sms, cudaStream_t s);

cudaError_t configure_linear_many(int dev);
int64_t linear_many_cycles(int T, int N, int KB, int dev, int sms);  // about how many its products take
cudaError_t launch_linear_many(const LinearArgs& l, const void* w, const void* x_codes, int64_t codes_stride, int dev, int sms, cudaStream_t s);

}  // namespace fw
