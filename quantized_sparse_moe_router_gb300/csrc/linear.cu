// Linear layers in 8 bits: argument checks and the choice of kernel.
#include <mutex>

#include "fp8.cuh"

using namespace fw;

static int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

static fw_status check_args(const fw_linear_fp8_args* a, bool pointers) {
  auto al = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!a) return set_error(FW_EINVAL, "fw_linear_fp8: null argument struct");
  if (a->T < 0 || a->N < 1 || a->K < 16 || a->K % 16) return set_error(FW_EINVAL, "fw_linear_fp8: need T >= 0, N >= 1 and K a positive multiple of 16");
  if (a->out_fp32 != 0 && a->out_fp32 != 1) return set_error(FW_EINVAL, "fw_linear_fp8: out_fp32 must be 0 or 1");
  if (a->T > (1 << 22) || a->N > (1 << 26)) return set_error(FW_EUNSUPPORTED, "fw_linear_fp8: at most 2^22 tokens and 2^26 outputs a call");
  if (!pointers || a->T == 0) return FW_OK;
  if (!a->x || !a->w || !a->w_scale || !a->out) return set_error(FW_EINVAL, "fw_linear_fp8: null pointer");
  if (!al(a->x, 16) || !al(a->w, 16) || !al(a->x_scale, 16) || !al(a->w_scale, 4) || !al(a->out, a->out_fp32 ? 4 : 2) || !al(a->status, 4))
    return set_error(FW_EINVAL, "fw_linear_fp8: x, x_scale and w need 16-byte alignment, the rest that of its elements");
  if (a->x_stride < a->K || a->x_stride % (a->x_scale ? 16 : 8) || a->out_stride < a->N)
    return set_error(FW_EINVAL, "fw_linear_fp8: token strides must cover the rows; x_stride a multiple of 8 (bf16) or 16 (codes) elements");
  if (a->x_scale && (a->x_scale_stride < a->T || a->x_scale_stride % 4))
    return set_error(FW_EINVAL, "fw_linear_fp8: x_scale_stride must cover T and be a multiple of 4 elements");
  return FW_OK;
}

// The current device and its SM count; its kernels are configured once.
static cudaError_t device_sms(int* device, int* sms) {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0, n = 0;
  if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> g(mu);
  if (!known[dev]) {
    cudaError_t e = configure_fp8_quantize();
    if (e == cudaSuccess) e = configure_linear_few(dev);
    if (e == cudaSuccess) e = configure_linear_many(dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    known[dev] = n;
  }
  *device = dev;
  *sms = known[dev];
  return cudaSuccess;
}

// The workspace: codes and scales of bf16 tokens that no kernel quantises itself.
static bool quantises_first(const fw_linear_fp8_args* a) { return !a->x_scale && !linear_few_quantises(a->T); }
static int64_t scale_stride(const fw_linear_fp8_args* a) { return round_up(a->T, 64); }
static int64_t codes_bytes(const fw_linear_fp8_args* a) { return round_up((int64_t)a->T * a->K, 256); }

// Up to 64 tokens the weights bound the call, and the kernel for few tokens reads them
// faster (64 x 7168 x 7168: 14.8 us against 15.7, 64 x 4096 x 4096: 8.7 against 10.0). With
// more both are estimated, by the cycles that the products of the one take and the blocks
// of K that an SM has in the other, 970 cycles each and 2,100 for the other's longer start
// and end (65 x 4096 x 2048: few 7.9 us, many 8.6; 130 x 7168 x 1024: 10.4 and 9.2; 257 x
// 4096 x 4096: 20.4 and 10.7; 400 x 1024 x 1024: 6.5 and 4.9).
static bool takes_many(const fw_linear_fp8_args* a, int dev, int sms) {
  const int KB = fp8_blocks(a->K);
  return a->T > 64 && linear_many_cycles(a->T, a->N, KB, dev, sms) <= linear_few_blocks(a->T, a->N, KB, dev, sms) * 970 + 2100;
}

extern "C" fw_status fw_linear_fp8_workspace(const fw_linear_fp8_args* a, int64_t* bytes) {
  if (!bytes) return set_error(FW_EINVAL, "fw_linear_fp8_workspace: null pointer");
  *bytes = 0;
  if (fw_status st = check_args(a, false); st != FW_OK) return st;
  if (a->T > 0 && quantises_first(a)) *bytes = codes_bytes(a) + scale_stride(a) * fp8_blocks(a->K) * 4;
  return FW_OK;
}

extern "C" fw_status fw_linear_fp8(const fw_linear_fp8_args* a, void* workspace, int64_t bytes, void* stream) {
  if (fw_status st = check_args(a, true); st != FW_OK) return st;
  if (a->T == 0) return FW_OK;
  int64_t need = 0;
  if (fw_status st = fw_linear_fp8_workspace(a, &need); st != FW_OK) return st;
  if (need && (!workspace || bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16))
    return set_error(FW_EINVAL, "fw_linear_fp8: the workspace is too small (see fw_linear_fp8_workspace) or not 16-byte aligned");
  if (fw_status st = check_device("fw_linear_fp8: needs an sm_103 device"); st != FW_OK) return st;
  int dev = 0, sms = 0;
  if (cudaError_t e = device_sms(&dev, &sms); e != cudaSuccess) return set_cuda_error(e, "fw_linear_fp8: setting the device up");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  LinearArgs l = {a->T, a->K, a->N, fp8_blocks(a->K), nullptr, 0, a->x_scale, a->x_scale_stride, a->w_scale, a->out, a->out_stride, a->out_fp32, a->status, 0};
  const void* codes = a->x;
  int64_t codes_stride = a->x_stride;
  cudaError_t e = cudaSuccess;
  if (quantises_first(a)) {
    float* scales = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + codes_bytes(a));
    e = launch_fp8_quantize(a->x, a->x_stride, a->T, a->K, workspace, scales, scale_stride(a), s);
    codes = workspace;
    codes_stride = a->K;
    l.x_scale = scales;
    l.x_scale_stride = scale_stride(a);
    l.x_alone = 1;
  } else if (!a->x_scale) {
    l.x = static_cast<const __nv_bfloat16*>(a->x);
    l.x_stride = a->x_stride;
  }
  if (e == cudaSuccess)
    e = takes_many(a, dev, sms) ? launch_linear_many(l, a->w, codes, codes_stride, dev, sms, s)
                           : launch_linear_few(l, a->w, codes, codes_stride, dev, sms, s);
  if (e != cudaSuccess) return set_cuda_error(e, "fw_linear_fp8: launch");
  return FW_OK;
}
