// What the attention kernels share: how a request's visible keys become
// stages of work, and the partial results that a split leaves behind.
#pragma once

#include "kvcache.cuh"

namespace fw {

constexpr int kStageKeys = 128;  // keys a kernel takes at a time: a whole number of pages
constexpr int kDecodeRows = 16;  // query rows (new tokens x heads of a group) the decode kernel takes at most

namespace dev {

constexpr float kLog2e = 1.4426950408889634f;

// The 128-key blocks that some of the query positions first .. S - 1 can see:
// `sink` blocks from 0, then the blocks lo .. end - 1.
struct Stages {
  int sink, lo, end;
  __device__ __forceinline__ int count() const { return sink + end - lo; }
  __device__ __forceinline__ int block(int s) const { return s < sink ? s : lo + s - sink; }
};
__device__ __forceinline__ Stages visible_stages(int S, int first, int window, int sinks) {
  Stages v;
  v.end = (S + kStageKeys - 1) / kStageKeys;
  const int lo = window ? ::max(0, ::max(0, first) + 1 - window) : 0;
  v.lo = lo / kStageKeys;
  v.sink = ::min((::min(sinks, lo) + kStageKeys - 1) / kStageKeys, v.lo);
  return v;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Whether a request's n new tokens from row q0 on are rows that the call has, no
// more than it allows for; reported if not.
__device__ __forceinline__ bool sound_queries(const fw_attn_q4_args& u, int q0, int n) {
  if (n >= 0 && n <= u.max_q && q0 >= 0 && q0 <= u.T - n) return true;
  raise(u.status, FW_KV_BAD_QUERIES);
  return false;
}

// Whether the query at position p sees key j (j >= 0).
__device__ __forceinline__ bool sees(int p, int j, int window, int sinks) {
  return j <= p && (window == 0 || j > p - window || j < sinks);
}

}  // namespace dev

// Partial results of one (request, key/value head, run of query rows) that
// several CTAs share: row-wise softmax maximum (in units of log2) and sum, and
// the unnormalised output. Part i is slot slot0 (i = 0) or slot1 + i step.
struct SplitRecord {
  int parts, slot0, slot1, step;  // parts = 0: nothing to join
  int rows, row0;                 // row n of a part is row m = row0 + n of the request:
  int token0, head0;              // token token0 + m / G, query head head0 + m % G
};

cudaError_t configure_decode_attn();
int64_t decode_workspace(const fw_attn_q4_args& a, int sms);
cudaError_t launch_attn_decode(const fw_attn_q4_args& a, void* workspace, int sms, cudaStream_t s);

cudaError_t configure_prefill_attn();
int64_t prefill_workspace(const fw_attn_q4_args& a, int sms);
// min_rows: requests of at most so many query rows are left to the decode kernel (0: none are)
cudaError_t launch_attn_prefill(const fw_attn_q4_args& a, int min_rows, void* workspace, int sms, cudaStream_t s);

// Joins the parts of `records` records; a slot holds rows_max rows of ml and o.
cudaError_t launch_attn_join(const fw_attn_q4_args& a, const SplitRecord* rec, const float* o, const float2* ml, int records,
                             int rows_max, cudaStream_t s);

}  // namespace fw
