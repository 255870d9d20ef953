// The norms after a block and before the next one, fused with the block's gate,
// the residual scale and the sum between them:
//
//   r = residual + scale * gate * y / sqrt(mean(y^2) + eps) * post_norm
//   h = r / sqrt(mean(r^2) + eps) * norm
//
// One pass: a row's values stay in registers between the two sums over it, so
// y and the residual are read once and r and h written once, which bounds many
// rows by HBM (4096 x 7168: 6.3 TB/s). A single row is bound by latency: its loads are
// all issued before anything waits for them. (Weights kept in shared memory with rows
// copied ahead into a ring of it, by one CTA an SM, were slower: 46 us against 37.)
//
// h may leave as 8-bit codes with a scale per 128 values (the linear layers'
// input): a thread holds eight neighbours, so a block is 16 neighbouring lanes.
#include <atomic>

#include "fp8.cuh"

namespace fw {
namespace {

using namespace dev;

constexpr int kMaxThreads = 1024, kMaxNormH = 32768;

// Sum over the row: a warp's own, or the CTA's (buf: one float a warp, used once).
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  v = warp_sum(v);
  if constexpr (!kWarp) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    v = warp_sum(lane < n ? buf[lane] : 0.f);
  }
  return v;
}

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  bf16x2_to_f32(v.x, f[0], f[1]);
  bf16x2_to_f32(v.y, f[2], f[3]);
  bf16x2_to_f32(v.z, f[4], f[5]);
  bf16x2_to_f32(v.w, f[6], f[7]);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]), bf16x2_bits(f[4], f[5]), bf16x2_bits(f[6], f[7]));
}
// Eight neighbouring floats of this lane, with one load or store where they are 32-byte
// aligned: the two halves of a warp's kilobyte one after the other take L1 twice the time,
// which bounded rows with weights (4096 x 7168 with norms on both sides: L1 at 74%).
template <bool kConst>
__device__ __forceinline__ void load8(const float* p, bool aligned, float (&f)[8]) {
  if (aligned) {
    if constexpr (kConst)
      asm("ld.global.nc.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
          : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
          : "l"(p));
    else  // (the residual, which may be written in place)
      asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                   : "l"(p)
                   : "memory");
  } else {
    const float4 a = kConst ? __ldg(reinterpret_cast<const float4*>(p)) : reinterpret_cast<const float4*>(p)[0];
    const float4 b = kConst ? __ldg(reinterpret_cast<const float4*>(p) + 1) : reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}
__device__ __forceinline__ void store8(float* p, bool aligned, const float (&f)[8]) {
  if (aligned) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]),
                 "f"(f[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// kVec: vectors of eight values a thread holds. kWarp: a warp a row, otherwise a
// CTA a row. kWide: residuals are fp32. kLoop: the CTA takes every gridDim.x-th row,
// and loads the next one once it has summed the row's parts.
// (1024 threads of four vectors with fp32 residuals, rows past 8192, have 64 registers
// each and keep 68 bytes of them in local memory.)
template <int kVec, bool kWarp, bool kWide, bool kLoop>
__global__ void __launch_bounds__(kWarp ? 256 : kVec <= 2 ? 512 : kMaxThreads, kWarp || kVec > 2 ? 1 : 2)
    norm_residual_kernel(const __grid_constant__ fw_norm_residual_args u) {
  __shared__ float s_sum[2][2][32];  // [odd turn][which sum]
  const int width = kWarp ? 32 : blockDim.x, l = kWarp ? threadIdx.x & 31 : threadIdx.x;
  int64_t row = kWarp ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const bool aligned = ((reinterpret_cast<uintptr_t>(u.norm) | reinterpret_cast<uintptr_t>(u.post_norm) |
                         (u.gate_fp32 && !u.gate_per_token ? reinterpret_cast<uintptr_t>(u.gate) : 0) |
                         (kWide ? reinterpret_cast<uintptr_t>(u.residual) | reinterpret_cast<uintptr_t>(u.residual_out) : 0)) & 31) == 0;
  uint4 yv[kVec], rv[kWide ? 1 : kVec];
  float rw[kWide ? kVec : 1][8];
  auto load = [&](bool in) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int at = 8 * (i * width + l);
      const bool has = in && at < u.H;
      yv[i] = has ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(u.y) + row * u.y_stride + at) : make_uint4(0u, 0u, 0u, 0u);
      const bool adds = has && u.residual;
      if constexpr (kWide) {
#pragma unroll
        for (int j = 0; j < 8; ++j) rw[i][j] = 0.f;
        if (adds) load8<false>(static_cast<const float*>(u.residual) + row * u.residual_stride + at, aligned, rw[i]);
      } else {
        rv[i] = adds ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(u.residual) + row * u.residual_stride + at) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  pdl_wait();
  pdl_launch_dependents();
  bool in = row < u.T;  // (kWarp: a warp past the last row goes along without loads or stores)
  load(in);
  for (int turn = 0;; turn ^= 1) {
    const int64_t now = row;
    float by = u.scale;
    if (u.gate && u.gate_per_token && in)
      by *= u.gate_fp32 ? __ldg(static_cast<const float*>(u.gate) + now * u.gate_stride)
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(u.gate)[now * u.gate_stride]);
    if (u.post_norm) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        float f[8];
        unpack8(yv[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
      }
      by *= rsqrtf(row_sum<kWarp>(sum, s_sum[turn][0]) / (float)u.H + u.eps);
    }
    float r[kVec][8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int at = 8 * (i * width + l);
      if (!in || at >= u.H) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = 0.f;
        continue;
      }
      float f[8], w[8];
      unpack8(yv[i], f);
      if constexpr (kWide) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = rw[i][j];
      } else {
        unpack8(rv[i], r[i]);
      }
      if (u.post_norm) {
        load8<true>(u.post_norm + at, aligned, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= w[j];
      }
      if (u.gate && !u.gate_per_token) {
        if (u.gate_fp32)
          load8<true>(static_cast<const float*>(u.gate) + now * u.gate_stride + at, aligned, w);
        else
          unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(u.gate) + now * u.gate_stride + at), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= w[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[i][j] = fmaf(f[j], by, r[i][j]);
        sum = fmaf(r[i][j], r[i][j], sum);
      }
    }
    const bool stores = in;
    bool more = false;
    if constexpr (kLoop) {
      row += gridDim.x;
      more = in = row < u.T;
      if (more) load(true);
    }
    if (u.residual_out && stores) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int at = 8 * (i * width + l);
        if (at >= u.H) continue;
        if constexpr (kWide) {
          store8(static_cast<float*>(u.residual_out) + now * u.residual_out_stride + at, aligned, r[i]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(u.residual_out) + now * u.residual_out_stride + at) = pack8(r[i]);
        }
      }
    }
    if (u.h || u.h_codes) {
      const float inv = u.norm ? rsqrtf(row_sum<kWarp>(sum, s_sum[turn][1]) / (float)u.H + u.eps) : 1.f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int at = 8 * (i * width + l);
        const bool has = stores && at < u.H;
        if (u.norm && has) {
          float w[8];
          load8<true>(u.norm + at, aligned, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) r[i][j] *= inv * w[j];
        }
        const uint4 out = pack8(r[i]);
        if (u.h && has) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(u.h) + now * u.h_stride + at) = out;
        if (u.h_codes) {  // (every lane takes part: past the row's end with zeros)
          float scale;
          const uint2 c = fp8_block_of_lanes(out, &scale);
          if (has) {
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(u.h_codes) + now * u.H + at) = c;
            if ((l & 15) == 0) u.h_scale[(at / kFp8Block) * u.h_scale_stride + now] = scale;
          }
        }
      }
    }
    if (!more) return;
  }
}

template <int kVec, bool kWarp, bool kLoop>
cudaError_t launch(const fw_norm_residual_args& u, unsigned grid, int threads, cudaStream_t s) {
  return u.residual_fp32 ? launch_dependent(norm_residual_kernel<kVec, kWarp, true, kLoop>, dim3(grid), dim3(threads), 0, s, u)
                         : launch_dependent(norm_residual_kernel<kVec, kWarp, false, kLoop>, dim3(grid), dim3(threads), 0, s, u);
}

cudaError_t sm_count(int* sms) {
  static std::atomic<int> known[64];  // of each device
  int dev = 0, n = 0;
  if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if ((n = known[dev].load()) == 0) {
    if (cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev); e != cudaSuccess) return e;
    known[dev].store(n);
  }
  *sms = n;
  return cudaSuccess;
}

}  // namespace
}  // namespace fw

using namespace fw;

extern "C" fw_status fw_norm_residual(const fw_norm_residual_args* u, void* stream) {
  auto al = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!u) return set_error(FW_EINVAL, "fw_norm_residual: null argument struct");
  if (u->T < 0 || u->H < 8 || u->H % 8) return set_error(FW_EINVAL, "fw_norm_residual: need T >= 0 and H a positive multiple of 8");
  if (u->H > kMaxNormH) return set_error(FW_EUNSUPPORTED, "fw_norm_residual: H is at most 32768");
  if (u->h_codes && u->H % 16) return set_error(FW_EINVAL, "fw_norm_residual: 8-bit codes need H a multiple of 16");
  if ((u->residual_fp32 | u->gate_fp32 | u->gate_per_token) & ~1) return set_error(FW_EINVAL, "fw_norm_residual: flags must be 0 or 1");
  if (!(u->eps >= 0.f)) return set_error(FW_EINVAL, "fw_norm_residual: eps must not be negative");
  if (u->T == 0) return FW_OK;
  if (!u->y || (!u->residual_out && !u->h && !u->h_codes) || (u->h_codes && !u->h_scale))
    return set_error(FW_EINVAL, "fw_norm_residual: null pointer (y, some output, and h_scale with h_codes are needed)");
  const int64_t H = u->H;
  if (u->y_stride < H || u->y_stride % 8 || (u->residual && (u->residual_stride < H || u->residual_stride % 8)) ||
      (u->residual_out && (u->residual_out_stride < H || u->residual_out_stride % 8)) || (u->h && (u->h_stride < H || u->h_stride % 8)))
    return set_error(FW_EINVAL, "fw_norm_residual: token strides must cover H and be multiples of 8 elements");
  if (u->h_codes && (u->h_scale_stride < u->T || u->h_scale_stride % 4))
    return set_error(FW_EINVAL, "fw_norm_residual: h_scale_stride must cover T and be a multiple of 4 elements");
  if (u->gate && (u->gate_per_token ? u->gate_stride < 0 : (u->gate_stride % 8 || (u->gate_stride != 0 && u->gate_stride < H))))
    return set_error(FW_EINVAL, "fw_norm_residual: gate_stride must be 0, or cover H and be a multiple of 8 (per token: not negative)");
  for (const void* p : {u->y, u->residual, u->gate_per_token ? nullptr : u->gate, (const void*)u->post_norm, (const void*)u->norm, (const void*)u->residual_out,
                        (const void*)u->h, (const void*)u->h_codes, (const void*)u->h_scale})
    if (!al(p, 16)) return set_error(FW_EINVAL, "fw_norm_residual: tensors need 16-byte alignment");
  if (!al(u->gate, u->gate_fp32 ? 4 : 2)) return set_error(FW_EINVAL, "fw_norm_residual: gate needs the alignment of its elements");
  if (fw_status st = check_device("fw_norm_residual: needs an sm_103 device"); st != FW_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int vecs = u->H / 8, T = u->T;
  cudaError_t e;
  if (vecs <= 128 && T > 1) {
    const int warps = 8, per = (vecs + 31) / 32;
    const unsigned grid = (unsigned)(((int64_t)T + warps - 1) / warps);
    e = per == 1   ? launch<1, true, false>(*u, grid, 32 * warps, s)
        : per == 2 ? launch<2, true, false>(*u, grid, 32 * warps, s)
                   : launch<4, true, false>(*u, grid, 32 * warps, s);
  } else {
    // One vector a thread up to 2048 columns, then two (at 4096, 4096 rows: 20 us against
    // 23), four past 8192. Rows that outnumber the SMs, and are long enough to wait for, are
    // looped over, two CTAs an SM and, with many, two turns of them (4096 x 7168: 42 -> 37
    // us, with norms on both sides and a gate 58 -> 48; 600 x 7168: 10 -> 8; 4096 x 2048: no
    // gain, 12.6).
    const int per = vecs <= 256 ? 1 : vecs <= 1024 ? 2 : 4;
    const int threads = ((vecs + per - 1) / per + 31) / 32 * 32;
    int sms = 0;
    if (cudaError_t err = sm_count(&sms); err != cudaSuccess) return set_cuda_error(err, "fw_norm_residual: the device's SM count");
    if (per == 2 && T > 2 * sms)
      e = launch<2, false, true>(*u, (unsigned)(T >= 8 * sms ? 4 * sms : 2 * sms), threads, s);
    else
      e = per == 1   ? launch<1, false, false>(*u, (unsigned)T, threads, s)
          : per == 2 ? launch<2, false, false>(*u, (unsigned)T, threads, s)
                     : launch<4, false, false>(*u, (unsigned)T, threads, s);
  }
  if (e != cudaSuccess) return set_cuda_error(e, "fw_norm_residual: launch");
  return FW_OK;
}
