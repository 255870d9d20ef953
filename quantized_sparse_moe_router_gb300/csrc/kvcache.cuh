// The 4-bit paged key/value cache: its page format, and what the kernels that
// write it, read it back and attend over it share.
//
// A page holds P consecutive positions of one request for every key/value
// head; the block of one (page, head) is contiguous:
//   K codes  [P][4 q][NB b] 32-bit words, NB = D / 32: dims 32 b + 8 q + i;
//            nibbles 0..3 hold i = 0, 2, 4, 6 and nibbles 4..7 i = 1, 3, 5, 7
//   K scales [P][NB] bf16
//   V codes  [P / 2][8 g][NB b] 32-bit words: dims 32 b + 4 g + i; nibbles 0..3
//            hold i = 0..3 of the even position, nibbles 4..7 of the odd one
//   V scales [P / 2][NB][2] bf16 (even, odd position)
// A value is scale * (code - 8). The orders are those of the matrix
// instructions' fragments: one shift and one AND-OR of a K word give two
// neighbouring dims of one position, of a V word one dim of two neighbouring
// positions -- the two operands that K^T q and V^T p want packed.
#pragma once

#include "internal.cuh"

namespace fw {

constexpr int kKvBlock = 32;  // values per 4-bit block

// Bytes of one (page, head) block.
__host__ __device__ inline int64_t kv_head_bytes(int page, int D) { return (int64_t)page * D * 9 / 8; }

// Byte offsets of the planes within one (page, head) block.
struct KvPlanes {
  int ks, vc, vs;
};
__host__ __device__ inline KvPlanes kv_planes(int page, int D) {
  const int codes = page * D / 2, scales = page * (D / kKvBlock) * 2;
  return {codes, codes + scales, 2 * codes + scales};
}

// Text of what is wrong with a cache's shape, or null; refusal of devices other than sm_103.
const char* kv_format_error(int n_kv, int page, int64_t n_pages);
fw_status check_device(const char* text);
// Records the error of a CUDA call that failed, with its name and text, for fw_moe_last_error; returns the status.
fw_status set_cuda_error(cudaError_t e, const char* what);

namespace dev {

// max / min that return NaN when either operand is (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// One bulk asynchronous copy shared -> global (16-byte aligned, size % 16 == 0), and the wait for this thread's.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_s2g_wait() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

// Sets bits of a caller's status word (may be null).
__device__ __forceinline__ void raise(int32_t* status, int bits) {
  if (status) atomicOr(status, bits);
}

}  // namespace dev
}  // namespace fw
