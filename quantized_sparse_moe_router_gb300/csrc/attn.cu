// Attention of a step's new tokens over the 4-bit paged cache.
//
//   out[t, h] = sum_j p_j v_j,  p = softmax over the visible j of scale * q[t, h] . k_j
//
// for request r's i-th new token at position p = seq_len - n_new + i; key j is
// visible when j <= p and (window == 0 or j > p - window or j < sinks).
#include <mutex>

#include "attn.cuh"

namespace fw {
namespace {

using namespace dev;

// One CTA per (token, query head), a thread per key of a 128-key tile, then a
// thread per dim: the definition with an online maximum and sum.
constexpr int kTile = 128;

template <int D>
__global__ void __launch_bounds__(kTile) attn_rows_kernel(fw_attn_q4_args a) {
  constexpr int NB = D / kKvBlock;
  __shared__ float s_q[D], s_p[kTile], s_red[kTile / 32];
  __shared__ int s_slot[kTile];  // byte offsets would not fit: page * page_size + place, or -1
  const int tid = threadIdx.x, t = blockIdx.x, h = blockIdx.y, hk = h / (a.n_q / a.n_kv);
  pdl_wait();
  pdl_launch_dependents();
  int lo = 0, hi = a.R;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a.q_start[m] <= t) lo = m; else hi = m;
  }
  const int r = lo;
  if (t < a.q_start[r] || t >= a.q_start[r + 1]) return;
  if ((a.q_start[r + 1] - a.q_start[r]) * (a.n_q / a.n_kv) <= kDecodeRows) return;  // the decode kernel's
  const int S = a.seq_lens[r], p = S - (a.q_start[r + 1] - t);
  for (int d = tid; d < D; d += kTile)
    s_q[d] = __bfloat162float(((const __nv_bfloat16*)a.q)[t * a.q_stride + h * D + d]) * a.scale;
  const int64_t hb = kv_head_bytes(a.page, D);
  const KvPlanes pl = kv_planes(a.page, D);
  const int w0 = a.window ? ::max(0, p + 1 - a.window) : 0;
  float m_run = -INFINITY, l_run = 0.f, acc[(D + kTile - 1) / kTile] = {};
  for (int j0 = 0; j0 <= p; j0 += kTile) {
    if (j0 + kTile <= w0 && j0 >= a.sinks) continue;
    const int j = j0 + tid;
    const bool see = j <= p && (j >= w0 || j < a.sinks);
    float x = -INFINITY;
    __syncthreads();
    s_slot[tid] = -1;
    if (see) {
      const int blk = j / a.page;
      int page = blk < a.max_blocks ? a.block_table[(int64_t)r * a.max_blocks + blk] : -1;
      if (page < 0 || page >= a.n_pages) {
        raise(a.status, FW_KV_BAD_SLOT);
      } else {
        const int at = j % a.page;
        s_slot[tid] = page * a.page + at;
        const uint8_t* base = (const uint8_t*)a.cache + ((int64_t)page * a.n_kv + hk) * hb;
        const uint32_t* k = reinterpret_cast<const uint32_t*>(base + at * (D / 2));
        const __nv_bfloat16* ks = reinterpret_cast<const __nv_bfloat16*>(base + pl.ks) + at * NB;
        x = 0.f;
        for (int b = 0; b < NB; ++b) {
          float s = 0.f;
          for (int q = 0; q < 4; ++q)
            for (int i = 0; i < 8; ++i)
              s += s_q[b * 32 + q * 8 + i] * (float)((int)(k[q * NB + b] >> (4 * (i / 2) + 16 * (i % 2)) & 15) - 8);
          x += s * __bfloat162float(ks[b]);
        }
      }
    }
    float m = x;
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((tid & 31) == 0) s_red[tid >> 5] = m;
    __syncthreads();
    m = fmaxf(m_run, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
    const float safe = m == -INFINITY ? 0.f : m, keep = __expf(m_run - safe);
    s_p[tid] = s_slot[tid] < 0 ? 0.f : __expf(x - safe);
    __syncthreads();
    m_run = m;
    l_run *= keep;
    for (int k = 0; k < kTile; ++k) l_run += s_p[k];
    for (int c = 0; c < (D + kTile - 1) / kTile; ++c) {
      const int d = c * kTile + tid;
      if (d >= D) break;
      acc[c] *= keep;
      const int b = d / 32, g = d % 32 / 4, i = d % 4;
      for (int k = 0; k < kTile; ++k) {
        const int slot = s_slot[k];
        if (slot < 0) continue;
        const int at = slot % a.page;
        const uint8_t* base = (const uint8_t*)a.cache + ((int64_t)(slot / a.page) * a.n_kv + hk) * hb;
        const uint32_t w = reinterpret_cast<const uint32_t*>(base + pl.vc + (at / 2) * D)[g * NB + b];
        const float vd = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base + pl.vs)[2 * ((at / 2) * NB + b) + (at & 1)]);
        acc[c] += s_p[k] * ((float)((int)(w >> (4 * i + 16 * (at & 1)) & 15) - 8) * vd);
      }
    }
  }
  for (int c = 0; c < (D + kTile - 1) / kTile; ++c) {
    const int d = c * kTile + tid;
    if (d < D) ((__nv_bfloat16*)a.out)[t * a.out_stride + h * D + d] = __float2bfloat16_rn(l_run != 0.f ? acc[c] / l_run : 0.f);
  }
}

}  // namespace
}  // namespace fw

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
  if ((int64_t)a->max_blocks * a->page > 0x7FFFFFFFll)
    return set_error(FW_EINVAL, "fw_attn_q4: need max_blocks * page < 2^31");
  // a request's 128-key units over all heads are counted in 32 bits, and so is a CTA's share of all (at least 152 CTAs)
  const int64_t units = ((int64_t)a->max_blocks * a->page / 128 + 2) * a->n_kv;
  if (units >= 1 << 30 || units / 128 * a->R >= 1 << 30)
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

// The current device's SM count, its kernels configured once; 0: no such device.
static int device_sms() {
  static std::mutex mu;
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> g(mu);
  if (!sms[dev]) {
    int n = 0;
    if (configure_attn_kernels() != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 0;
    sms[dev] = n;
  }
  return sms[dev];
}

static bool has_decode(const fw_attn_q4_args* a) { return a->n_q / a->n_kv <= kDecodeRows; }

extern "C" fw_status fw_attn_q4_workspace(const fw_attn_q4_args* a, int64_t* bytes) {
  if (!bytes) return set_error(FW_EINVAL, "fw_attn_q4_workspace: null pointer");
  *bytes = 0;
  if (fw_status st = check_args(a, false); st != FW_OK) return st;
  if (a->R == 0 || a->T == 0 || a->max_q == 0) return FW_OK;
  if (fw_status st = check_device("fw_attn_q4: needs an sm_103 device"); st != FW_OK) return st;
  const int sms = device_sms();
  if (!sms) return set_error(FW_ECUDA, "fw_attn_q4: the device could not be set up");
  if (has_decode(a)) *bytes = decode_workspace(*a, sms);
  return FW_OK;
}

extern "C" fw_status fw_attn_q4(const fw_attn_q4_args* a, void* workspace, int64_t bytes, void* stream) {
  if (fw_status st = check_args(a, true); st != FW_OK) return st;
  if (a->R == 0 || a->T == 0 || a->max_q == 0) return FW_OK;
  int64_t need = 0;
  if (fw_status st = fw_attn_q4_workspace(a, &need); st != FW_OK) return st;
  if (need && (!workspace || bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16))
    return set_error(FW_EINVAL, "fw_attn_q4: the workspace is too small (see fw_attn_q4_workspace) or not 16-byte aligned");
  const int sms = device_sms(), G = a->n_q / a->n_kv;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (has_decode(a)) e = launch_attn_decode(*a, workspace, sms, s);
  if (e == cudaSuccess && (int64_t)a->max_q * G > kDecodeRows)
    e = dev::launch_dependent(a->D == 64 ? attn_rows_kernel<64> : attn_rows_kernel<128>, dim3(a->T, a->n_q), dim3(kTile), 0, s, *a);
  if (e != cudaSuccess) return set_error(FW_ECUDA, "fw_attn_q4: launch failed");
  return FW_OK;
}
