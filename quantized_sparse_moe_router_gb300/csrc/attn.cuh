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

// Whether the query at position p sees key j (j >= 0).
__device__ __forceinline__ bool sees(int p, int j, int window, int sinks) {
  return j <= p && (window == 0 || j > p - window || j < sinks);
}

}  // namespace dev

// Partial result of one (request, key/value head) that several CTAs share:
// row-wise softmax maximum (in units of log2) and sum, and the unnormalised
// output. Slot 2 c + i: CTA c's first (i = 0) or a later (i = 1) segment.
struct SplitRecord {  // of the CTA that holds the first part
  int parts, slot0, cta0, rows;  // parts = 0: nothing to join; part i > 0 is slot 2 (cta0 + i)
  int token0, head0, group, pad; // row n is token token0 + n / group, query head head0 + n % group
};

cudaError_t configure_attn_kernels();
int64_t decode_workspace(const fw_attn_q4_args& a, int sms);
cudaError_t launch_attn_decode(const fw_attn_q4_args& a, void* workspace, int sms, cudaStream_t s);

}  // namespace fw
