// Attention of a step's new tokens over the 4-bit paged cache: argument checks
// and the choice of kernels.
//
//   out[t, h] = sum_j p_j v_j,  p = softmax over the visible j of scale * q[t, h] . k_j
//
// for request r's i-th new token at position p = seq_len - n_new + i; key j is
// visible when j <= p and (window == 0 or j > p - window or j < sinks).
//
// Two kernels share a call's requests by the query rows (new tokens x heads
// that share a key/value head) each of them brings: up to kDecodeRows go to
// the decode kernel, more to the prefill kernel. Which requests those are only
// the device knows, so a call that may hold both kinds launches both.
#include <algorithm>
#include <mutex>

#include "attn.cuh"

using namespace fw;

static fw_status check_args(const fw_attn_q4_args* a, bool pointers) {
  auto al = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!a) return set_error(FW_EINVAL, "fw_attn_q4: null argument struct");
  if (a->D != 64 && a->D != 128) return set_error(FW_EUNSUPPORTED, "fw_attn_q4: D must be 64 or 128");
  if (const char* e = kv_format_error(a->n_kv, a->page, a->n_pages)) return set_error(FW_EINVAL, e);
  if (a->n_q < 1 || a->n_q % a->n_kv || a->n_q / a->n_kv > 128)
    return set_error(FW_EINVAL, "fw_attn_q4: n_q must be n_kv times 1..128");
  if (a->R < 0 || a->R > (1 << 20) || a->T < 0 || a->max_q < 0 || a->max_q > a->T || a->max_blocks < 1)
    return set_error(FW_EINVAL, "fw_attn_q4: need 0 <= R <= 2^20, 0 <= max_q <= T and max_blocks >= 1");
  if (a->window < 0 || a->sinks < 0) return set_error(FW_EINVAL, "fw_attn_q4: window and sinks must not be negative");
  // (positions are rounded up to whole stages in 32 bits)
  if ((int64_t)a->max_blocks * a->page > 0x7FFFFFFFll - kStageKeys)
    return set_error(FW_EINVAL, "fw_attn_q4: need max_blocks * page < 2^31 - 128");
  // a request's 128-key units over all heads are counted in 32 bits, and so is
  // what a CTA takes of all of them: shares are equal in cost, and a pair's
  // fixed cost is six units, so no share is more than seven times the mean
  const int64_t units = ((int64_t)a->max_blocks * a->page / 128 + 2) * a->n_kv;
  if (units >= 1 << 30 || units / 32 * a->R >= 1 << 30)
    return set_error(FW_EUNSUPPORTED, "fw_attn_q4: R block-table rows of max_blocks pages are beyond any cache");
  if (!(a->scale > 0.f) || a->scale > 3e38f) return set_error(FW_EINVAL, "fw_attn_q4: scale must be positive and finite");
  if (!pointers || a->R == 0 || a->T == 0 || a->max_q == 0) return FW_OK;
  if (!a->q || !a->out || !a->cache || !a->block_table || !a->q_start || !a->seq_lens)
    return set_error(FW_EINVAL, "fw_attn_q4: null pointer");
  if (!al(a->q, 16) || !al(a->out, 16) || !al(a->cache, 16) || !al(a->block_table, 4) || !al(a->q_start, 4) ||
      !al(a->seq_lens, 4) || !al(a->status, 4))
    return set_error(FW_EINVAL, "fw_attn_q4: q, out and cache need 16-byte, the rest 4-byte alignment");
  const int64_t w = (int64_t)a->n_q * a->D;
  if (a->q_stride < w || a->out_stride < w || a->q_stride % 8 || a->out_stride % 8)
    return set_error(FW_EINVAL, "fw_attn_q4: token strides must cover the heads and be multiples of 8 elements");
  return FW_OK;
}

// The current device's SM count; its kernels are configured once.
static cudaError_t device_sms(int* sms) {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0, n = 0;
  if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> g(mu);
  if (!known[dev]) {
    cudaError_t e = configure_decode_attn();
    if (e == cudaSuccess) e = configure_prefill_attn();
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    known[dev] = n;
  }
  *sms = known[dev];
  return cudaSuccess;
}

// Whether the decode kernel runs. Not where no request can bring few enough
// rows, nor where all seem to bring the same, too many (one request, or T rows
// for R requests of max_q): the prefill kernel then takes whatever there is.
static bool may_decode(const fw_attn_q4_args* a) {
  const int G = a->n_q / a->n_kv;
  const bool many = (int64_t)a->max_q * G > kDecodeRows;
  return G <= kDecodeRows && !(many && (a->R == 1 || (int64_t)a->R * a->max_q == a->T));
}
static bool may_prefill(const fw_attn_q4_args* a) { return (int64_t)a->max_q * (a->n_q / a->n_kv) > kDecodeRows; }

extern "C" fw_status fw_attn_q4_workspace(const fw_attn_q4_args* a, int64_t* bytes) {
  if (!bytes) return set_error(FW_EINVAL, "fw_attn_q4_workspace: null pointer");
  *bytes = 0;
  if (fw_status st = check_args(a, false); st != FW_OK) return st;
  if (a->R == 0 || a->T == 0 || a->max_q == 0) return FW_OK;
  if (fw_status st = check_device("fw_attn_q4: needs an sm_103 device"); st != FW_OK) return st;
  int sms = 0;
  if (cudaError_t e = device_sms(&sms); e != cudaSuccess) return set_cuda_error(e, "fw_attn_q4: setting the device up");
  // (the kernels of a call run one after the other: they share the workspace)
  if (may_decode(a)) *bytes = decode_workspace(*a, sms);
  if (may_prefill(a)) *bytes = std::max(*bytes, prefill_workspace(*a, sms));
  return FW_OK;
}

extern "C" fw_status fw_attn_q4(const fw_attn_q4_args* a, void* workspace, int64_t bytes, void* stream) {
  if (fw_status st = check_args(a, true); st != FW_OK) return st;
  if (a->R == 0 || a->T == 0 || a->max_q == 0) return FW_OK;
  int64_t need = 0;
  if (fw_status st = fw_attn_q4_workspace(a, &need); st != FW_OK) return st;
  if (need && (!workspace || bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16))
    return set_error(FW_EINVAL, "fw_attn_q4: the workspace is too small (see fw_attn_q4_workspace) or not 16-byte aligned");
  int sms = 0;
  if (cudaError_t e = device_sms(&sms); e != cudaSuccess) return set_cuda_error(e, "fw_attn_q4: setting the device up");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (may_decode(a)) e = launch_attn_decode(*a, workspace, sms, s);
  if (e == cudaSuccess && may_prefill(a)) e = launch_attn_prefill(*a, may_decode(a) ? kDecodeRows : 0, workspace, sms, s);
  if (e != cudaSuccess) return set_cuda_error(e, "fw_attn_q4: launch");
  return FW_OK;
}
