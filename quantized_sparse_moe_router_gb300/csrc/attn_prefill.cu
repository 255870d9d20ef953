// Attention for requests that bring many query rows (prompts and chunks of
// them): a dense contraction per (request, key/value head), on the tcgen05
// tensor cores.
//
//   S = Q K^T,  P = 2^(scale S - m),  O = sum over key tiles of P V,  out = O / l
//
// The rows of a head's group are packed (row = new token x G + head in the
// group), so a key/value head's tiles are unpacked once for all its query
// heads. A CTA owns 256 rows as two 128-row tiles, and walks the 128-key tiles
// that they see. While one tile is in its softmax the tensor core works on the
// other: per row tile the steps S(i) -> P(i) -> O(i) are serial, S and P share
// tensor-memory columns, and the issue order PV(i), QK(i + 1) of one warp is
// all the ordering that needs.
//
// 16 warps: 0-3 and 4-7 softmax of row tile 0 and 1 (a thread a row: no
// shuffles; S in 128 registers), 8-11 unpack the 4-bit codes to 16-bit operand
// tiles (K by keys, V transposed by dims, both K-major with the 128-byte
// swizzle), 12 issues the
// MMAs, 13 copies pages (one bulk copy each). Bound by
// the tensor core at head dims of 128, by the softmax's instructions at 64.
//
// Tensor memory: S0 | S1 | O0 | O1, 128 columns each; P (bf16) over the first
// 64 columns of its S. Shared memory: Q, a ring of three unpacked tiles taken in
// the order K0 V0 K1 V1 ..., a ring of three packed tiles.
#include <initializer_list>

#include "attn.cuh"
#include "tcgen05.cuh"

namespace fw {
namespace {

using namespace dev;

constexpr int kRowTile = 128, kBlockRows = 2 * kRowTile;
constexpr int kThreads = 512;
constexpr int kDeqWarp0 = 8, kMmaWarp = 12, kLoadWarp = 13;
constexpr int kPacked = 3, kTiles = 3, kHave = 8, kPoison = 4;
constexpr int kSoftmaxRegs = 184, kOtherRegs = 72;  // of 128 a thread at launch
constexpr uint32_t kTmemCols = 512;
constexpr float kMost = 1048576.f;  // a row's maximum moves only when a tile's sum of p passes this

template <int D>
struct Cfg {
  static constexpr int NB = D / kKvBlock;
  static constexpr uint32_t QBytes = kRowTile * D * 2;        // one row tile: [D / 64] panels of [128 rows][128 B]
  static constexpr uint32_t TileBytes = kStageKeys * D * 2;   // K: as Q; V: [2] panels of 64 keys, [D dims][128 B]
  static constexpr uint32_t PackedBytes = kStageKeys * D * 9 / 8;
  static constexpr uint32_t SmemBytes = 2 * QBytes + kTiles * TileBytes + kPacked * PackedBytes + 1024;
};

struct PrefillArgs {
  fw_attn_q4_args u;
  int splits;        // CTAs that share a block's key tiles
  int min_rows;      // requests of at most so many rows are not this kernel's
  int blocks;        // blocks of 256 rows at most (grid = blocks * n_kv * splits)
  float* o;          // splits > 1: [blocks * n_kv * splits][256][D]
  float2* ml;        // [blocks * n_kv * splits][256]
  SplitRecord* rec;  // [blocks * n_kv]
  float scale_log2;
};

__device__ __forceinline__ uint32_t bf16x2_op_sub136(uint32_t x) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x43084308u));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_op_mul(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// Keys go to f16, values to bf16. A key d (c - 8) has at most 8 + 3 significant
// bits, so f16 holds it exactly (scores are then exact up to the fp32 sums,
// however large); what f16 lacks in range is made up by powers of two: a
// query row is scaled to a magnitude of 1..2, and all keys by 2^-6, which
// leaves them 4 10^6 at the top and an absolute error of 2^-19 at the bottom.
// Values keep bf16's range; they and the probabilities are rounded once.
constexpr float kKeyScale = 1.f / 64.f;

// nibbles 2 k + {0, 1} (and + 4) of a word, shifted to the low byte of each
// half -> two f16 pairs (c - 8) d: the upper nibble stands for 16 c as it is,
// and takes d / 16
__device__ __forceinline__ void unpack_f16(uint32_t w, uint32_t mask, uint32_t mask4, uint32_t d, uint32_t d16, uint32_t& lo, uint32_t& hi) {
  uint32_t x, y;
  asm("lop3.b32 %0, %1, %2, 0x64006400, 0xEA;" : "=r"(x) : "r"(w), "r"(mask));        // 1024 + c
  asm("lop3.b32 %0, %1, %2, 0x64006400, 0xEA;" : "=r"(y) : "r"(w), "r"(mask4));   // 1024 + 16 c
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(0x64086408u));               // - 1032
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(y), "r"(0x64806480u));               // - 1152
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(d));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(d16));
}
__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// nibbles at bit `shift` of a word's halves -> (c - 8) * d, rounded once to bf16
__device__ __forceinline__ uint32_t unpack(uint32_t w, int shift, uint32_t mask, uint32_t d) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, 0x43004300, 0xEA;" : "=r"(r) : "r"(w >> shift), "r"(mask));
  return bf16x2_op_mul(bf16x2_op_sub136(r), d);
}
__device__ __forceinline__ bool finite_bf16(uint32_t bits) { return (bits & 0x7F80u) != 0x7F80u; }

// A bounded wait with its loop in place (where warps change their register
// share a call would need a register split of its own) and without a suspend
// hint: a thread that sleeps on one wakes about 1000 cycles after the barrier
// flips, which the chain of softmax and products would pay four times a tile.
__device__ __forceinline__ bool mbar_wait_inline(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(PrefillArgs a) {
  using C = Cfg<D>;
  constexpr int NB = C::NB;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t packed_full[kPacked], packed_empty[kPacked], tile_full[kTiles], tile_empty[kTiles];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], o_full, q_full;
  __shared__ uint32_t s_tmem, s_have[kHave];
  __shared__ __align__(4) uint8_t s_flag[kPoison][4];       // per unpacking warp: some scale of V is not finite
  __shared__ uint8_t s_poison[kPoison][kStageKeys];  // then: the key's blocks (bits) that are not
  __shared__ int s_scan[kThreads / 32], s_found[4];
  __shared__ float s_qscale[kBlockRows];  // powers of two the query rows were divided by
  const fw_attn_q4_args& u = a.u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = u.n_q / u.n_kv;
  const int z = blockIdx.x % a.splits, pair = blockIdx.x / a.splits, head = pair % u.n_kv;
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = base;
  uint8_t* sT = sQ + 2 * C::QBytes;
  uint8_t* sP = sT + kTiles * C::TileBytes;
  pdl_wait();
  pdl_launch_dependents();

  // Which block of which request: the blocks in descending order of their
  // place, so that a prompt's later rows, which see the most keys, start first.
  int total = 0, want = -1;
  for (int pass = 0; pass < 2; ++pass) {
    int sum = 0;
    for (int r0 = 0; r0 < u.R; r0 += kThreads) {
      const int r = r0 + tid;
      int n = 0, q0 = 0, nb = 0;
      if (r < u.R) {
        q0 = u.q_start[r];
        n = u.q_start[r + 1] - q0;
        if (n * (long long)G > a.min_rows && q0 >= 0 && q0 <= u.T - n) nb = (int)((n * (long long)G + kBlockRows - 1) / kBlockRows);
      }
      int inc = nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += x;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = inc;
      __syncthreads();
      int before = sum + inc - nb;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        sum += s_scan[w];
      }
      if (want >= before && want < before + nb) {
        s_found[0] = r;
        s_found[1] = want - before;
        s_found[2] = n;
        s_found[3] = q0;
      }
      if (pass == 0 && r0 + kThreads >= u.R) {
        total = sum;
        want = total - 1 - pair / u.n_kv;
        // one chunk holds everybody: no second pass
        if (u.R <= kThreads && want >= before && want < before + nb) {
          s_found[0] = r;
          s_found[1] = want - before;
          s_found[2] = n;
          s_found[3] = q0;
        }
      }
    }
    if (want < 0 || u.R <= kThreads) break;
  }
  if (want < 0) {  // fewer blocks than the host had to allow for
    if (a.splits > 1 && z == 0 && tid == 0) a.rec[pair].parts = 0;
    return;
  }
  __syncthreads();
  const int r = s_found[0], row0 = s_found[1] * kBlockRows, n_new = s_found[2], tok0 = s_found[3];
  const int rows = ::min(kBlockRows, n_new * G - row0), row_tiles = rows > kRowTile ? 2 : 1;
  int S = u.seq_lens[r];
  if (S > u.max_blocks * u.page) {
    S = u.max_blocks * u.page;
    if (tid == 0) raise(u.status, FW_KV_BAD_SLOT);
  }
  const int first = S - n_new + row0 / G, last = S - n_new + (row0 + rows - 1) / G;  // positions of the block's rows
  const Stages v = visible_stages(::max(last + 1, 0), first, u.window, u.sinks);
  const int lo_key = u.window ? ::max(0, ::max(0, first) + 1 - u.window) : 0;
  const int n_all = v.count(), i0 = (int)((long long)n_all * z / a.splits), n_t = (int)((long long)n_all * (z + 1) / a.splits) - i0;
  const int64_t part = blockIdx.x;
  if (a.splits > 1 && z == 0 && tid == 0) {
    SplitRecord rec;
    rec.parts = a.splits;
    rec.slot0 = rec.slot1 = pair * a.splits;
    rec.step = 1;
    rec.rows = rows;
    rec.token0 = tok0;
    rec.row0 = row0;
    rec.head0 = head * G;
    a.rec[pair] = rec;
  }

  if (tid == 0) {
    for (int i = 0; i < kPacked; ++i) {
      mbar_init(&packed_full[i], 1);
      mbar_init(&packed_empty[i], 4);
    }
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&tile_full[i], 4);
      mbar_init(&tile_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    mbar_init(&o_full, 1);
    mbar_init(&q_full, 8);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const KvPlanes pl = kv_planes(u.page, D);
  const uint32_t hb = (uint32_t)kv_head_bytes(u.page, D);
  const int page_shift = __ffs(u.page) - 1;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {  // by a whole warp, or one thread alone
    if (ok && !mbar_wait_inline(bar, parity)) {
      ok = false;
      raise(u.status, FW_KV_TIMEOUT);
    }
    return ok;
  };

  if (warp < kDeqWarp0) {
    // ------------------------------------------------ softmax: a thread a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int t = warp >> 2, row = t * kRowTile + (warp & 3) * 32 + lane;
    // this thread's share of Q into shared memory: 16 bytes a lane, rows of a
    // token side by side (all 256 rows: those past the last are zeros)
    for (int e = tid; e < kBlockRows * (D / 8); e += kDeqWarp0 * 32) {
      const int qr = e / (D / 8), c = e % (D / 8), n = row0 + qr;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (qr < rows)
        w = *reinterpret_cast<const uint4*>((const __nv_bfloat16*)u.q + (int64_t)(tok0 + n / G) * u.q_stride + (head * G + n % G) * D + 8 * c);
      float x[8], most = 0.f;
      bf16x2_to_f32(w.x, x[0], x[1]);
      bf16x2_to_f32(w.y, x[2], x[3]);
      bf16x2_to_f32(w.z, x[4], x[5]);
      bf16x2_to_f32(w.w, x[6], x[7]);
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(x[j]));
#pragma unroll
      for (int j = 1; j < D / 8; j <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, j));
      // 2^e of the largest magnitude; rows of zeros, tiny rows and rows that are not finite as they are
      const uint32_t ex = __float_as_uint(most) & 0x7F800000u;
      const bool plain = ex < (64u << 23) || ex == 0x7F800000u;
      const float down = plain ? 1.f : __uint_as_float((254u << 23) - ex);
      if (c == 0) s_qscale[qr] = plain ? 1.f : __uint_as_float(ex);
      w = make_uint4(f16x2_bits(x[0] * down, x[1] * down), f16x2_bits(x[2] * down, x[3] * down), f16x2_bits(x[4] * down, x[5] * down),
                     f16x2_bits(x[6] * down, x[7] * down));
      const int rr = qr % kRowTile;
      *reinterpret_cast<uint4*>(sQ + (qr / kRowTile) * C::QBytes + (c / 8) * (kRowTile * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = w;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full);
    if (t < row_tiles) {
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_cols = tmem + lanes + t * 128, o_cols = tmem + lanes + 256 + t * 128;
      const int p = row < rows ? S - n_new + (row0 + row) / G : -1;
      float mz = 0.f, l = 0.f, scale = 0.f;
      bool first_max = true;  // none was taken yet
      uint32_t poison = 0;
      int key_before = 0;
      // blocks of V that are not finite in keys this row sees (the tile whose product is in O by now)
      auto check_poison = [&](int i, int key0) {
        const uint32_t flags = *reinterpret_cast<volatile uint32_t*>(s_flag[i % kPoison]);
        if (flags == 0) return;
        for (int c = 0; c < kStageKeys; ++c)
          if ((flags >> (8 * (c / 32)) & 1) && sees(p, key0 + c, u.window, u.sinks)) poison |= s_poison[i % kPoison][c];
      };
      for (int i = 0; i < n_t; ++i) {
        const int key0 = v.block(i0 + i) * kStageKeys;
        wait(&s_full[t], i & 1);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        tc_fence_after();
        // (the first score tells that every row of Q and its scale were written)
        if (i == 0) scale = a.scale_log2 * (1.f / kKeyScale) * s_qscale[row];
        uint32_t s[128];
        tmem_ld128(s_cols, s);
        if (i > 0) check_poison(i - 1, key_before);
        key_before = key0;
        const uint32_t have = s_have[i % kHave];
        if (key0 + kStageKeys - 1 > first || (u.window && key0 < last + 1 - u.window) || have != 0xFF) {
          const int hi = p - key0, lo = u.window ? hi - u.window : -1, sk = u.sinks - key0;  // sees: c <= hi, c > lo or c < sk
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (!(c <= hi && (c > lo || c < sk) && (have >> (c / 16) & 1))) s[c] = 0xFF800000u;  // -inf
        }
        // P and its sum against the maximum as last taken; both are exact to
        // their rounding whatever their magnitude, so it only has to move
        // when a tile's sum shows that some p is past kMost (or none was taken)
        auto weights = [&]() {
          const f2 sc = f2_pack(scale, scale), mm = f2_pack(-mz, -mz);
          f2 sum = f2_pack(0.f, 0.f), sum2 = sum;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float x, y;
              f2_unpack(f2_fma(f2_pack_bits(s[32 * c + 2 * j], s[32 * c + 2 * j + 1]), sc, mm), x, y);
              x = exp2_fast(x);
              y = exp2_fast(y);
              if (j & 1) sum2 = f2_add(sum2, f2_pack(x, y)); else sum = f2_add(sum, f2_pack(x, y));
              pk[j] = bf16x2_bits(x, y);
            }
            tmem_st16(s_cols + 16 * c, pk);
          }
          float x, y;
          f2_unpack(f2_add(sum, sum2), x, y);
          return x + y;
        };
        float sum = first_max ? 0.f : weights();
        if (__any_sync(0xFFFFFFFFu, first_max || sum > kMost)) {
          float top = -INFINITY, top2 = -INFINITY;
#pragma unroll
          for (int c = 0; c < 128; c += 4) {
            top = fmaxf(top, fmaxf(__uint_as_float(s[c]), __uint_as_float(s[c + 1])));
            top2 = fmaxf(top2, fmaxf(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])));
          }
          float up = fmaf(fmaxf(top, top2), scale, -mz);
          // a first maximum is taken as it is, a later one only moves up
          if (!first_max) up = fmaxf(up, 0.f);
          const bool none = up == -INFINITY;
          const float keep = first_max ? 0.f : exp2_fast(-up);
          if (!none) {
            mz += up;
            l *= keep;
            first_max = false;
          }
          if (i > 0) {  // O holds the tiles before: S(i) came after their product
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {  // 16 columns at a time: S holds 128 registers
              uint32_t o[16];
              tmem_ld16(o_cols + c, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = none ? o[j] : __float_as_uint(__uint_as_float(o[j]) * keep);
              tmem_st16(o_cols + c, o);
            }
          }
          sum = weights();
        }
        l += sum;
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      // ---------------------------------------------- out = O / l
      if (n_t > 0) {
        wait(&o_full, 0);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok) check_poison(n_t - 1, key_before);
      }
      const int n = row0 + row;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (a.splits > 1 && row < rows) a.ml[part * kBlockRows + row] = make_float2(first_max ? -INFINITY : mz, l);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (n_t > 0 && ok) {
          tmem_ld32(o_cols + c, o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0;
        }
        if (poison >> (c / kKvBlock) & 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0x7FC00000u;  // NaN
        }
        if (row >= rows) continue;
        if (a.splits > 1) {
          if (n_t == 0) continue;  // the join leaves an empty part alone
          float* dst = a.o + (part * kBlockRows + row) * D + c;
#pragma unroll
          for (int j = 0; j < 32; j += 4) *reinterpret_cast<uint4*>(dst + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        } else {
          __nv_bfloat16* dst = (__nv_bfloat16*)u.out + (int64_t)(tok0 + n / G) * u.out_stride + (head * G + n % G) * D + c;
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = bf16x2_bits(__uint_as_float(o[j + 2 * k]) * inv, __uint_as_float(o[j + 2 * k + 1]) * inv);
            *reinterpret_cast<uint4*>(dst + j) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------ unpack 4-bit codes to operand tiles
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    const int w = warp - kDeqWarp0;
    uint32_t mask;
    asm volatile("mov.u32 %0, 0x000F000F;" : "=r"(mask));
    const int key = 32 * w + lane, at = key & (u.page - 1);      // K: a lane a key
    const uint32_t blk_k = (key >> page_shift) * hb;
    for (int i = 0; i < n_t; ++i) {
      const int key0 = v.block(i0 + i) * kStageKeys;
      const uint8_t* pk = sP + (i % kPacked) * C::PackedBytes;
      wait(&packed_full[i % kPacked], (i / kPacked) & 1);
      // ---- K
      uint32_t seq = 2 * i;
      wait(&tile_empty[seq % kTiles], ((seq / kTiles) & 1) ^ 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      {
        uint8_t* tile = sT + (seq % kTiles) * C::TileBytes;
        const uint8_t* codes = pk + blk_k + at * (D / 2);
        uint32_t d[NB], d16[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float x = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(pk + blk_k + pl.ks)[at * NB + b] << 16) * kKeyScale;
          d[b] = f16x2_bits(x, x);
          d16[b] = f16x2_bits(x * 0.0625f, x * 0.0625f);
        }
        // the 16-byte chunk 4 b + q of this key lies at ((4 (b & 1) + q) ^ (key & 7)) in panel b / 2
        uint8_t* row = tile + key * 128;
        const int x4 = (key & 4) << 4;
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          const int q = (qq + (NB == 4 ? lane >> 1 : lane >> 2)) & 3;  // (the reads of 8 lanes fall into different banks)
          uint8_t* at_q = row + ((q ^ (key & 3)) << 4);
          uint32_t x[NB];
          if constexpr (NB == 4) {
            const uint4 c4 = *reinterpret_cast<const uint4*>(codes + q * 16);
            x[0] = c4.x; x[1] = c4.y; x[2] = c4.z; x[3] = c4.w;
          } else {
            const uint2 c2 = *reinterpret_cast<const uint2*>(codes + q * 8);
            x[0] = c2.x; x[1] = c2.y;
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint4 o;
            unpack_f16(x[b], mask, mask << 4, d[b], d16[b], o.x, o.y);
            unpack_f16(x[b] >> 8, mask, mask << 4, d[b], d16[b], o.z, o.w);
            *reinterpret_cast<uint4*>(at_q + (b / 2) * (kStageKeys * 128) + (x4 ^ ((b & 1) << 6))) = o;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tile_full[seq % kTiles]);
      // ---- V: this warp's 32 keys as four 8-key chunks; a lane four dims of one block
      seq = 2 * i + 1;
      wait(&tile_empty[seq % kTiles], ((seq / kTiles) & 1) ^ 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      {
        uint8_t* tile = sT + (seq % kTiles) * C::TileBytes;
        // byte offset of a key pair's codes and scales within the packed tile
        auto codes_at = [&](int kp) { return ((2 * kp) >> page_shift) * hb + pl.vc + (kp & (u.page / 2 - 1)) * D; };
        auto scales_at = [&](int kp) { return ((2 * kp) >> page_shift) * hb + pl.vs + (kp & (u.page / 2 - 1)) * (NB * 4); };
        // scales that must not enter the product: keys past the last or of a
        // missing page (whatever is there), and what is not finite (noted for
        // the rows that see it). Half a pair's blocks to a lane.
        const uint32_t have = s_have[i % kHave] >> (2 * w) & 3;
        bool odd_tile = have != 3 || key0 + 32 * w + 32 > S;
        uint32_t bad0 = 0, bad1 = 0;  // blocks of the even and the odd key
        {
          const int kp = 16 * w + lane / 2;
          const uint32_t at_s = scales_at(kp);
#pragma unroll
          for (int k = 0; k < NB / 2; ++k) {
            const int b = (lane & 1) * (NB / 2) + k;
            const uint32_t sc = *reinterpret_cast<const uint32_t*>(pk + at_s + b * 4);
            if (!finite_bf16(sc & 0xFFFFu)) bad0 |= 1u << b;
            if (!finite_bf16(sc >> 16)) bad1 |= 1u << b;
          }
          const bool there = have >> (lane / 16) & 1;
          if (!there || key0 + 2 * kp >= S) bad0 = 0;
          if (!there || key0 + 2 * kp + 1 >= S) bad1 = 0;
          const bool some = __any_sync(0xFFFFFFFFu, (bad0 | bad1) != 0);
          if (some) {
            bad0 |= __shfl_xor_sync(0xFFFFFFFFu, bad0, 1);
            bad1 |= __shfl_xor_sync(0xFFFFFFFFu, bad1, 1);
            if ((lane & 1) == 0) {
              s_poison[i % kPoison][2 * kp] = (uint8_t)bad0;
              s_poison[i % kPoison][2 * kp + 1] = (uint8_t)bad1;
            }
            odd_tile = true;
          }
          __syncwarp();
          if (lane == 0) s_flag[i % kPoison][w] = some;
        }
        constexpr int Lanes = 8 * NB, Chunks = 32 / Lanes;  // lanes of a pair's words; chunks side by side in a warp
        const int word = lane % Lanes, b = word % NB, g = word / NB;
#pragma unroll
        for (int cc = 0; cc < 4; cc += Chunks) {
          const int c = 4 * w + cc + lane / Lanes;  // chunk of 8 keys
          uint32_t x[4], d[4];
          const uint8_t* in_x = pk + codes_at(4 * c) + word * 4;  // (a chunk's four pairs are one page's)
          const uint8_t* in_d = pk + scales_at(4 * c) + b * 4;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[k] = *reinterpret_cast<const uint32_t*>(in_x + k * D);
            d[k] = *reinterpret_cast<const uint32_t*>(in_d + k * (NB * 4));
          }
          if (odd_tile) {
            const bool there = s_have[i % kHave] >> (c / 2) & 1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = key0 + 8 * c + 2 * k;
              if (!there || j >= S || !finite_bf16(d[k] & 0xFFFFu)) d[k] &= 0xFFFF0000u;
              if (!there || j + 1 >= S || !finite_bf16(d[k] >> 16)) d[k] &= 0xFFFFu;
            }
          }
          uint8_t* col = tile + (c / 8) * (D * 128) + (32 * b + 4 * g) * 128;
          const int c4 = (c & 7) ^ ((g & 1) << 2);  // ((dim & 7) = 4 (g & 1) + j)
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {
            const int j = (jj + (NB == 4 ? b : 2 * b + (g >> 1))) & 3;  // (the writes of 8 lanes fall into different banks)
            *reinterpret_cast<uint4*>(col + j * 128 + ((c4 ^ j) << 4)) =
                make_uint4(unpack(x[0], 4 * j, mask, d[0]), unpack(x[1], 4 * j, mask, d[1]), unpack(x[2], 4 * j, mask, d[2]),
                           unpack(x[3], 4 * j, mask, d[3]));
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&tile_full[seq % kTiles]);
        mbar_arrive(&packed_empty[i % kPacked]);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kMmaWarp) {
      // ---------------------------------------------- MMA issuer
      // The warp stays together and elects a lane for the MMAs only: their
      // descriptors are then uniform, and their issue fast enough. One issuer
      // and a fixed order keep the two row tiles half a period apart: with an
      // issuer each they fall into step, and softmax and products take turns
      // instead of overlapping.
      // (a value shuffled from lane 0 is uniform for the compiler, too)
      const uint32_t q0 = __shfl_sync(0xFFFFFFFFu, sw128_desc_lo(smem_u32(sQ)), 0);
      const uint32_t t0 = __shfl_sync(0xFFFFFFFFu, sw128_desc_lo(smem_u32(sT)), 0);
      const uint32_t cols = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      auto qk = [&](int t, uint32_t seq, bool last_use) {
        const uint32_t k0 = t0 + (seq % kTiles) * (C::TileBytes >> 4), a0 = q0 + t * (C::QBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = ((k / 4) * (kRowTile * 128) + (k % 4) * 32) >> 4;  // (both tiles have 128 rows)
            mma_ss_lo(cols + t * 128, a0 + at, k0 + at, idesc_f16(kRowTile, kStageKeys), k != 0);
          }
          mma_commit(&s_full[t]);
          if (last_use) mma_commit(&tile_empty[seq % kTiles]);
        }
        __syncwarp();
      };
      auto pv = [&](int t, uint32_t seq, bool more, bool last_use) {
        const uint32_t v0 = t0 + (seq % kTiles) * (C::TileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kStageKeys / 16; ++k)
            mma_ts_lo(cols + 256 + t * 128, cols + t * 128 + k * 8, v0 + (((k / 4) * (D * 128) + (k % 4) * 32) >> 4),
                      idesc_bf16(kRowTile, D), more || k != 0);
          if (last_use) mma_commit(&tile_empty[seq % kTiles]);
        }
        __syncwarp();
      };
      auto ready = [&](uint64_t* bar, uint32_t parity) {
        wait(bar, parity);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        return ok;
      };
      auto tile_ready = [&](uint32_t seq) { return ready(&tile_full[seq % kTiles], (seq / kTiles) & 1); };
      if (n_t > 0 && ready(&q_full, 0) && tile_ready(0)) {
        for (int t = 0; t < row_tiles; ++t) qk(t, 0, t == row_tiles - 1);
        for (int i = 0; i < n_t && ok; ++i) {
          const bool next = i + 1 < n_t;
          if (!tile_ready(2 * i + 1)) break;
          for (int t = 0; t < row_tiles; ++t) {
            if (!ready(&p_full[t], i & 1)) break;
            pv(t, 2 * i + 1, i > 0, t == row_tiles - 1);
            if (next) {
              if (t == 0 && !tile_ready(2 * i + 2)) break;
              qk(t, 2 * i + 2, t == row_tiles - 1);
            }
          }
        }
        // every MMA issued has finished before tensor memory is read or released
        if (elect_one()) mma_commit(&o_full);
        __syncwarp();
        mbar_wait_inline(&o_full, 0);
      }
    } else if (warp == kLoadWarp) {
      // ---------------------------------------------- pages, one to a lane
      int id = 0;
      auto look = [&](int i) {
        const int key = v.block(i0 + i) * kStageKeys + (lane << page_shift);
        const bool need = lane < (kStageKeys >> page_shift) && key <= last && (key + u.page > lo_key || key < u.sinks);
        if (need) id = u.block_table[(int64_t)r * u.max_blocks + (key >> page_shift)];
        return need;
      };
      bool need = n_t > 0 && look(0);
      int issued = 0;
      for (int i = 0; i < n_t; ++i) {
        bool copy = need;
        if (copy && (id < 0 || id >= u.n_pages)) {
          copy = false;
          raise(u.status, FW_KV_BAD_SLOT);
        }
        const int page = id, slot = i % kPacked;
        if (i + 1 < n_t) need = look(i + 1);  // in flight during this tile
        const uint32_t got = __ballot_sync(0xFFFFFFFFu, copy);
        wait(&packed_empty[slot], ((i / kPacked) & 1) ^ 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if (lane == 0) {
          uint32_t have = 0;  // a page's bit, for each 16 keys of it
#pragma unroll
          for (int k = 0; k < kStageKeys / 16; ++k) have |= (got >> ((k * 16) >> page_shift) & 1) << k;
          s_have[i % kHave] = have;
          mbar_arrive_expect_tx(&packed_full[slot], (uint32_t)__popc(got) * hb);
        }
        __syncwarp();
        if (copy)
          bulk_g2s(sP + slot * C::PackedBytes + lane * hb, (const uint8_t*)u.cache + ((int64_t)page * u.n_kv + head) * hb, hb,
                   &packed_full[slot]);
        issued = i + 1;
      }
      // copies still in flight after an abandoned wait land before the CTA leaves
      if (!ok)
        for (int j = ::max(0, issued - kPacked); j < issued; ++j) mbar_wait_inline(&packed_full[j % kPacked], (j / kPacked) & 1);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

int prefill_blocks(const fw_attn_q4_args& a) {
  // each request's last block may be partial; no more requests than tokens
  return (int)((int64_t)a.T * (a.n_q / a.n_kv) / kBlockRows + ::min(a.R, a.T));
}

// CTAs per block of rows: as many as fill the SMs once, and no more than there
// can be key tiles.
int prefill_splits(const fw_attn_q4_args& a, int sms) {
  const int64_t ctas = (int64_t)prefill_blocks(a) * a.n_kv;
  const int64_t tiles = ((int64_t)a.max_blocks * a.page + kStageKeys - 1) / kStageKeys;
  return (int)::max((int64_t)1, ::min(tiles, sms / ctas));
}

}  // namespace

cudaError_t configure_prefill_attn() {
  // the warps' register shares (setmaxnreg) must fit what the launch gives
  // the CTA, or the growing ones would wait for ever
  for (const void* k : {(const void*)attn_prefill_kernel<64>, (const void*)attn_prefill_kernel<128>}) {
    cudaFuncAttributes f;
    const cudaError_t e = cudaFuncGetAttributes(&f, k);
    if (e != cudaSuccess) return e;
    if (f.numRegs * kThreads < kSoftmaxRegs * 256 + kOtherRegs * 256) return cudaErrorInvalidDeviceFunction;
  }
  cudaError_t e = cudaFuncSetAttribute(attn_prefill_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<64>::SmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_prefill_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<128>::SmemBytes);
  return e;
}

int64_t prefill_workspace(const fw_attn_q4_args& a, int sms) {
  const int64_t pairs = (int64_t)prefill_blocks(a) * a.n_kv, splits = prefill_splits(a, sms);
  return splits == 1 ? 0 : pairs * sizeof(SplitRecord) + pairs * splits * kBlockRows * (a.D * 4 + 8);
}

cudaError_t launch_attn_prefill(const fw_attn_q4_args& a, int min_rows, void* workspace, int sms, cudaStream_t s) {
  PrefillArgs d;
  d.u = a;
  d.min_rows = min_rows;
  d.splits = prefill_splits(a, sms);
  d.blocks = prefill_blocks(a);
  const int64_t pairs = (int64_t)d.blocks * a.n_kv;
  if (pairs * d.splits > 0x7FFFFFFF) return cudaErrorInvalidValue;
  d.rec = static_cast<SplitRecord*>(workspace);
  d.o = reinterpret_cast<float*>(d.rec + pairs);
  d.ml = reinterpret_cast<float2*>(d.o + pairs * d.splits * kBlockRows * a.D);
  d.scale_log2 = a.scale * kLog2e;
  cudaError_t e = launch_dependent(a.D == 64 ? attn_prefill_kernel<64> : attn_prefill_kernel<128>, dim3((unsigned)(pairs * d.splits)),
                                   dim3(kThreads), a.D == 64 ? Cfg<64>::SmemBytes : Cfg<128>::SmemBytes, s, d);
  if (e == cudaSuccess && d.splits > 1) e = launch_attn_join(a, d.rec, d.o, d.ml, (int)pairs, kBlockRows, s);
  return e;
}

}  // namespace fw
