// Linear layers in 8 bits for many tokens: a matrix product bound by the tensor
// cores.
//
//   out[t][n] = sum_b xs[b][t] ws[n / 128][b] (sum_{k in block b} xc[t][k] wc[n][k])
//
// Two CTAs of a cluster work on one tile of 256 tokens by 256 outputs with one
// instruction (cta_group::2): each holds half of the tokens and half of the
// outputs' weights, so an SM takes in 128 + 128 rows a block of K for the
// products of 128 x 256. (A CTA by itself would need 128 + 256, more than L2
// gives an SM while its tensor core runs.)
//
// The tensor core adds up within a block of 128 along K; the block's scales are
// any fp32 numbers, so eight warps take each block's sums out of tensor memory,
// scale them and add them in registers (a thread a token and half of the columns)
// while the next block's products run into the other buffer. That is half of
// what the products take: one packed multiply-add for two sums.
//
// Where tiles are too few for the pairs, a cluster of two or four pairs takes one, each
// with a part of K, and joins the sums in their order through distributed shared memory.
//
// Warps: 0, 2 and 3 copy, 1 issues the products (the first CTA's for both), 4-11
// scale and add (tensor-memory quarter = warp % 4). Tiles are taken in turn by CTA pairs
// that stay, all 256 or all 128 outputs wide (see cut_of). Results leave through shared
// memory by TMA while the next tile runs.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fp8.cuh"
#include "pair.cuh"
#include "tcgen05.cuh"

namespace fw {
namespace {

using namespace dev;

constexpr int kTokRows = 128;                // tokens of a CTA
constexpr int kEpiWarps = 8;
constexpr int kFirstEpi = 4;                 // warps 0-3: copies and products
constexpr int kThreads = (kFirstEpi + kEpiWarps) * 32;
// registers of the first warpgroup and of the other two, of 168 a thread at launch: 128 x 56 + 256 x 224 = 384 x 168
constexpr int kFewRegs = 56, kEpiRegs = 224;
constexpr int kJoin = 16;                    // columns that a pair joins at once, where pairs share a tile
constexpr uint32_t kOutBytes = 32 * 128;     // a warp's staging: 32 rows of 128 bytes

constexpr uint32_t kXBytes = kTokRows * kFp8Block;
// The tokens' scales of a block come with the copies of the block before (a unit's
// first ones with its own), into a slot of their own: once a block's products are
// done the next block's scales are there, and can be read before they are needed.
// (Fetched by the warps that use them their latency bounded the kernel; held further
// ahead in registers, the sums spilled.) A block's copies start when the products
// Stages blocks before are done, which were issued when the sums of Acc blocks before those
// had been read: a slot comes round again after more.
constexpr int kSlots = 16;
constexpr uint32_t kScaleBytes = kTokRows * 4;
constexpr uint32_t kFixed = 1024 + kEpiWarps * kOutBytes + kSlots * kScaleBytes + 512;  // alignment, staging, scales, barriers
// Tiles are 256 outputs wide, or 128 where that leaves fewer pairs idle.
template <int kCols>
struct Many {
  static constexpr uint32_t WBytes = kCols / 2 * kFp8Block, StageBytes = kXBytes + WBytes;
  static constexpr int Stages = (int)((227 * 1024 - kFixed) / StageBytes);
  static constexpr int Acc = 512 / kCols;        // buffers of sums in tensor memory
  static constexpr uint32_t SmemBytes = 1024 + Stages * StageBytes + kEpiWarps * kOutBytes + kSlots * kScaleBytes;
  // (see kSlots)
  static_assert(kSlots > Stages + Acc + 1, "a slot of scales is read before it is filled again");
};

struct ManyArgs {
  LinearArgs l;
  int tiles_t, tiles_n;
  int tiles;
  int split;                                 // pairs that share a tile, each a part of K (more than one: a pair has one tile)
  int by_tma;                                // results leave by TMA (aligned rows that end with 16 bytes)
};

__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kSw128DescHi)
      : "memory");
}
// (No release at cluster scope: what the arrival follows are loads from tensor
// memory, complete by then; a fence for the rest of memory took 2000 cycles a block.)
__device__ __forceinline__ void arrive_at(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory"); }

// Columns of this thread's tensor-memory lane: on their way, and there.
__device__ __forceinline__ void tmem_ld_start(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
                 "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                 "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// (there as well: with the one that was waited for)
__device__ __forceinline__ void tmem_ld_there(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]),
                    "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// acc += r * s, two columns at a time.
template <int N>
__device__ __forceinline__ void add_scaled(f2* acc, const uint32_t (&r)[N], f2 s) {
#pragma unroll
  for (int j = 0; j < N; j += 2) acc[j / 2] = f2_fma(f2_pack_bits(r[j], r[j + 1]), s, acc[j / 2]);
}

// The same by two scales one after the other.
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <int N>
__device__ __forceinline__ void add_scaled(f2* acc, const uint32_t (&r)[N], f2 first, f2 then) {
#pragma unroll
  for (int j = 0; j < N; j += 2) acc[j / 2] = f2_fma(f2_mul(f2_pack_bits(r[j], r[j + 1]), first), then, acc[j / 2]);
}

// Tile i of 256 tokens and kCols outputs: neighbours share tokens in runs of kRun
// token tiles, whose weights are then read close together.
constexpr int kRun = 8;
template <int kCols>
__device__ __forceinline__ void tile_at(const ManyArgs& a, int i, int* t0, int* n0) {
  const int band = i / (kRun * a.tiles_n), first = band * kRun, rows = ::min(kRun, a.tiles_t - first), in = i - first * a.tiles_n;
  const int tn = in / rows;
  *t0 = (first + in - tn * rows) * 2 * kTokRows;
  *n0 = tn * kCols;
}

// 32 rows, a lane's row in `sum`, of kJoin outputs from `col` on: 16 bytes a lane and store
// where rows are aligned, otherwise through shared memory, two rows a store.
template <bool kFp32>
__device__ __forceinline__ void put_share(const LinearArgs& l, int aligned, const f2 (&sum)[kJoin / 2], int row0, int col, int lane, float* stage) {
  float v[kJoin];
#pragma unroll
  for (int j = 0; j < kJoin / 2; ++j) f2_unpack(sum[j], v[2 * j], v[2 * j + 1]);
  const int64_t size = kFp32 ? 4 : 2;
  uint8_t* out = static_cast<uint8_t*>(l.out);
  if (aligned && col + kJoin <= l.N) {
    if (row0 + lane >= l.T) return;
    uint4* to = reinterpret_cast<uint4*>(out + ((int64_t)(row0 + lane) * l.out_stride + col) * size);
    if constexpr (kFp32) {
#pragma unroll
      for (int j = 0; j < kJoin / 4; ++j)
        to[j] = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
    } else {
#pragma unroll
      for (int j = 0; j < kJoin / 8; ++j)
        to[j] = make_uint4(bf16x2_bits(v[8 * j], v[8 * j + 1]), bf16x2_bits(v[8 * j + 2], v[8 * j + 3]), bf16x2_bits(v[8 * j + 4], v[8 * j + 5]),
                           bf16x2_bits(v[8 * j + 6], v[8 * j + 7]));
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < kJoin; ++j) stage[lane * (kJoin + 1) + j] = v[j];
  __syncwarp();
  const int c = lane % kJoin;
#pragma unroll
  for (int r = lane / kJoin; r < 32; r += 32 / kJoin) {
    if (row0 + r >= l.T || col + c >= l.N) continue;
    const int64_t to = (int64_t)(row0 + r) * l.out_stride + col + c;
    if constexpr (kFp32)
      static_cast<float*>(l.out)[to] = stage[r * (kJoin + 1) + c];
    else
      static_cast<__nv_bfloat16*>(l.out)[to] = __float2bfloat16_rn(stage[r * (kJoin + 1) + c]);
  }
}

// kShare: a.split pairs share a tile.
template <int kCols, bool kFp32, bool kShare>
__global__ void __launch_bounds__(kThreads, 1) linear_many_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                                                                  const __grid_constant__ CUtensorMap map_s,
                                                                  const __grid_constant__ CUtensorMap map_o, const ManyArgs a) {
  using M = Many<kCols>;
  constexpr int kStages = M::Stages, kAcc = M::Acc, kMine = kCols / 2;  // kMine: columns of a thread
  // Columns that a load takes out of tensor memory, and loads at once: with 256 outputs, whose
  // buffers come round sooner than they are read, four (1024 x 7168 x 4096 27.0 -> 26.2 us);
  // with 128 one (four: 2048 x 2048 x 5120 22.7 -> 24.0).
  constexpr int kChunk = 16, kLoads = kCols == 256 ? 4 : 1;
  constexpr bool kAsk = kCols == 128;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], acc_full[kAcc], acc_empty[kAcc];
  __shared__ uint32_t s_tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = kShare ? a.split : 1, rank = blockIdx.x & 1, part = kShare ? (blockIdx.x >> 1) % split : 0;
  const int pair = (blockIdx.x >> 1) / split, pairs = (gridDim.x >> 1) / split;
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* ring = smem_raw + pad;                          // [kStages][tokens 128 x 128, weights 128 x 128]
  uint8_t* s_out = ring + kStages * M::StageBytes;           // [kEpiWarps][32 rows][128 bytes]
  float* s_scale = reinterpret_cast<float*>(s_out + kEpiWarps * kOutBytes);  // [kSlots][kTokRows]
  const LinearArgs& l = a.l;
  const int b0 = (int)((int64_t)l.KB * part / split), KB = (int)((int64_t)l.KB * (part + 1) / split) - b0;  // this pair's blocks of K

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kEpiWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are set up, and their tensor memory is there
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  bool ok = true;
  if (!l.x_alone || warp == 0 || warp == 3) pdl_wait();
  pdl_launch_dependents();

  if (warp == 0 || warp == 2 || warp == 3) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    // Warp 0 copies the tokens, 2 the weights, 3 the scales: a copy takes its warp some
    // 100 cycles to start. They stay together and elect a lane for it.
    const uint32_t first_full = in_cta(full, 2 * part);
    uint32_t i = 0, s = 0, phase = 1;
    for (int tile = pair; tile < a.tiles && ok; tile += pairs) {
      int t0, n0;
      tile_at<kCols>(a, tile, &t0, &n0);
      t0 += rank * kTokRows;
      n0 += rank * (kCols / 2);
      for (int b = 0; b < KB; ++b, ++i) {
        if (!(ok = __all_sync(0xFFFFFFFFu, wait_inline(&empty[s], phase)))) {
          raise(l.status, FW_KV_TIMEOUT);
          break;
        }
        if (elect_one()) {
          uint8_t* st = ring + s * M::StageBytes;
          const uint32_t bar = first_full + s * 8;
          if (warp == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (M::StageBytes + kScaleBytes * ((b == 0) + (b + 1 < KB))));
            tma_pair(st, &map_x, (b0 + b) * kFp8Block, t0, bar);
          } else if (warp == 2) {
            tma_pair(st + kXBytes, &map_w, (b0 + b) * kFp8Block, n0, bar);
          } else {
            if (b == 0) tma_pair(s_scale + i % kSlots * kTokRows, &map_s, t0, b0 + b, bar);
            if (b + 1 < KB) tma_pair(s_scale + (i + 1) % kSlots * kTokRows, &map_s, t0, b0 + b + 1, bar);
          }
        }
        __syncwarp();
        if (++s == kStages) s = 0, phase ^= 1;
      }
    }
    // (after a wait that gave up) both CTAs' copies in flight land before either leaves
    if (!ok && rank == 0 && warp == 0)
      for (uint32_t j = i > kStages ? i - kStages : 0; j < i; ++j) wait_inline(&full[j % kStages], (j / kStages) & 1);
    if constexpr (kShare) cluster_sync();  // (the parts' sums)
  } else if (warp == 1) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (rank == 0) {
      // The warp stays together and elects a lane for the products: their
      // descriptors are then uniform (a value shuffled from lane 0 is, for the compiler).
      const uint32_t ring_lo = __shfl_sync(0xFFFFFFFFu, sw128_desc_lo(smem_u32(ring)), 0), cols0 = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const int mine = pair < a.tiles ? (a.tiles - pair + pairs - 1) / pairs : 0;
      const uint32_t blocks = (uint32_t)mine * KB;
      uint32_t i = 0, s = 0, s_phase = 0;
      for (; i < blocks; ++i) {
        const uint32_t c = i % kAcc, c_phase = ((i / kAcc) & 1) ^ 1;
        // (both are asked at once: an answer takes some 70 cycles)
        const bool f = mbar_test(&full[s], s_phase), e = mbar_test(&acc_empty[c], c_phase);
        if (!__all_sync(0xFFFFFFFFu, f && e)) {
          ok = wait_inline(&full[s], s_phase) && wait_inline(&acc_empty[c], c_phase);
          if (!__all_sync(0xFFFFFFFFu, ok)) {
            raise(l.status, FW_KV_TIMEOUT);
            break;
          }
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t x = ring_lo + s * (M::StageBytes >> 4), w = x + (kXBytes >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_pair(cols0 + c * kCols, x + 2 * k, w + 2 * k, idesc_e4m3(2 * kTokRows, kCols), k != 0);
          commit_pair(&acc_full[c], 2 * part);
          commit_pair(&empty[s], 2 * part);
        }
        __syncwarp();
        if (++s == kStages) s = 0, s_phase ^= 1;
      }
      if (i > 0) wait_inline(&acc_full[(i - 1) % kAcc], ((i - 1) / kAcc) & 1);  // no product outlives the tensor memory
    }
    if constexpr (kShare) cluster_sync();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int q = warp & 3, half = (warp - kFirstEpi) >> 2;
    const uint32_t from0 = tmem + ((uint32_t)(32 * q) << 16);
    uint8_t* stage = s_out + (warp - kFirstEpi) * kOutBytes;
    const uint32_t first_empty = in_cta(acc_empty, 2 * part);
    uint32_t i = 0;
    for (int tile = pair; tile < a.tiles && ok; tile += pairs) {
      int t0, n0;
      tile_at<kCols>(a, tile, &t0, &n0);
      const int row0 = t0 + rank * kTokRows + 32 * q, col0 = n0 + half * kMine;
      // (columns of a thread lie in one block of 128 outputs; past the last one there is nothing to scale)
      const float* ws = l.w_scale + (int64_t)::min(col0 / kFp8Block, (l.N - 1) / kFp8Block) * l.KB + b0;
      f2 acc[kMine / 2];
#pragma unroll
      for (int j = 0; j < kMine / 2; ++j) acc[j] = 0ull;
      float w_now = 0.f, w_next = lane < KB ? __ldg(ws + lane) : 0.f;  // the weights' scales of 32 blocks, one a lane
      // Whatever a block waits for beside its sums is asked for while the block before
      // is being added: its barrier, its scale. (Done in turn that took a third of the time.)
      bool ready = false;
      float scale = 0.f;
      const auto add_blocks = [&](auto joined, int b, int end) {
        for (; b < end; ++b, ++i) {
          const uint32_t c = i % kAcc;
          if (!ready && !__all_sync(0xFFFFFFFFu, wait_inline(&acc_full[c], (i / kAcc) & 1))) {
            raise(l.status, FW_KV_TIMEOUT);
            ok = false;
            break;
          }
          tc_fence_after();
          if (b == 0) scale = s_scale[i % kSlots * kTokRows + 32 * q + lane] * __shfl_sync(0xFFFFFFFFu, w_now, 0);
          const uint32_t from = from0 + c * (2 * kMine) + half * kMine;
          const f2 s2 = f2_pack(scale, scale);
          uint32_t v[kLoads][kChunk];
#pragma unroll
          for (int j0 = 0; j0 < kMine; j0 += kLoads * kChunk) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) tmem_ld_start(from + j0 + j * kChunk, v[j]);
            if (j0 == (kLoads > 1 ? 0 : kMine - 2 * kChunk)) {
              const bool more = b + 1 < KB;
              if constexpr (kAsk) ready = __all_sync(0xFFFFFFFFu, more && mbar_test(&acc_full[(i + 1) % kAcc], ((i + 1) / kAcc) & 1));
              scale = more ? s_scale[(i + 1) % kSlots * kTokRows + 32 * q + lane] : 0.f;
              scale *= __shfl_sync(0xFFFFFFFFu, (b + 1) % 32 ? w_now : w_next, (b + 1) % 32);
            }
            tmem_ld_done(v[0]);
#pragma unroll
            for (int j = 1; j < kLoads; ++j) tmem_ld_there(v[j]);
            if (j0 + kLoads * kChunk == kMine) {  // (all of this warp's sums are in registers)
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_at(first_empty + c * 8);
            }
            if (joined) {
#pragma unroll
              for (int j = 0; j < kLoads; ++j) add_scaled(acc + (j0 + j * kChunk) / 2, v[j], s2);
            } else {  // (the block's own scale is still in its slot, see kSlots)
              const float f = s_scale[i % kSlots * kTokRows + 32 * q + lane], w = __shfl_sync(0xFFFFFFFFu, w_now, b % 32);
#pragma unroll
              for (int j = 0; j < kLoads; ++j) add_scaled(acc + (j0 + j * kChunk) / 2, v[j], f2_pack(w, w), f2_pack(f, f));
            }
          }
        }
      };
      for (int b = 0; b < KB && ok; b += 32) {
        w_now = w_next;
        w_next = b + 32 + lane < KB ? __ldg(ws + b + 32 + lane) : 0.f;
        // (see scales_join; 256 wide, with 64 columns to a branch, one loop is faster: 1500 x 5120 x
        // 5120 35.8 us against 43.9, 8192 x 4096 x 4096 97 against 114; 128 wide it is the slower)
        const bool joined = __all_sync(0xFFFFFFFFu, b + lane >= KB || scales_join(w_now));
        if constexpr (kLoads > 1)
          add_blocks(joined, b, ::min(KB, b + 32));
        else if (joined)
          add_blocks(std::true_type(), b, ::min(KB, b + 32));
        else
          add_blocks(std::false_type(), b, ::min(KB, b + 32));
      }
      // A tile that pairs share: each leaves its sums in its ring, which nothing reads or fills
      // any more, and joins, in the pairs' order, a share of every thread's columns.
      if constexpr (kShare) {
        const int at = threadIdx.x - kFirstEpi * 32, share = kMine / kJoin / split;
        float4* mine = reinterpret_cast<float4*>(ring) + at;  // [kMine / 4][a thread]
        if (ok) {
#pragma unroll
          for (int j = 0; j < kMine / 4; ++j) {
            if (j * 4 / kJoin / share == part) continue;
            float4 v;
            f2_unpack(acc[2 * j], v.x, v.y);
            f2_unpack(acc[2 * j + 1], v.z, v.w);
            mine[j * kEpiWarps * 32] = v;
          }
        }
        cluster_sync();
        if (!ok) break;
#pragma unroll
        for (int j0 = 0; j0 < kMine; j0 += kJoin) {
          if (j0 / kJoin / share != part) continue;
          f2 sum[kJoin / 2];
#pragma unroll
          for (int j = 0; j < kJoin / 2; ++j) sum[j] = 0ull;
          for (int p = 0; p < split; ++p) {
            const uint32_t from = in_cta(mine, 2 * p + rank);
#pragma unroll
            for (int j = 0; j < kJoin / 4; ++j) {
              f2 lo = acc[j0 / 2 + 2 * j], hi = acc[j0 / 2 + 2 * j + 1];
              if (p != part) {
                const float4 v = ld_cta(from + (j0 / 4 + j) * kEpiWarps * 32 * 16);
                lo = f2_pack(v.x, v.y), hi = f2_pack(v.z, v.w);
              }
              sum[2 * j] = f2_add(sum[2 * j], lo);
              sum[2 * j + 1] = f2_add(sum[2 * j + 1], hi);
            }
          }
          put_share<kFp32>(l, a.by_tma, sum, row0, col0 + j0, lane, reinterpret_cast<float*>(stage));
        }
        continue;
      }
      if (!ok) break;
      // 32 rows of 128 bytes at a time, the 16-byte chunk j of a row at j ^ (row % 8): the tensor map's swizzle
      constexpr int kStep = kFp32 ? 32 : 64;
#pragma unroll
      for (int j0 = 0; j0 < kMine; j0 += kStep) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint4 o;
          if constexpr (kFp32) {
            const f2 p = acc[(j0 + 4 * j) / 2], r = acc[(j0 + 4 * j) / 2 + 1];
            o = make_uint4((uint32_t)p, (uint32_t)(p >> 32), (uint32_t)r, (uint32_t)(r >> 32));
          } else {
            uint32_t w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              float lo, hi;
              f2_unpack(acc[(j0 + 8 * j) / 2 + h], lo, hi);
              w[h] = bf16x2_bits(lo, hi);
            }
            o = make_uint4(w[0], w[1], w[2], w[3]);
          }
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = o;
        }
        if (a.by_tma) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row0 < l.T && col0 + j0 < l.N) tma_out(&map_o, stage, col0 + j0, row0);
        } else {  // (rows of no alignment: neighbouring lanes write neighbouring outputs)
          __syncwarp();
          const int rows = ::min(32, l.T - row0);
          for (int r = 0; r < rows; ++r) {
            const int64_t at = (int64_t)(row0 + r) * l.out_stride + col0 + j0;
#pragma unroll
            for (int h = 0; h < kStep / 32; ++h) {
              const int c = lane + 32 * h;
              if (col0 + j0 + c >= l.N) continue;
              if constexpr (kFp32)
                static_cast<float*>(l.out)[at + c] = *reinterpret_cast<const float*>(stage + r * 128 + ((c / 4 ^ (r & 7)) << 4) + c % 4 * 4);
              else
                static_cast<uint16_t*>(l.out)[at + c] = *reinterpret_cast<const uint16_t*>(stage + r * 128 + ((c / 8 ^ (r & 7)) << 4) + c % 8 * 2);
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves, or gives its tensor memory back, while the other's products or signals reach it
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <int kCols, bool kFp32, bool kShare>
cudaError_t launch(const LinearArgs& l, const void* w, const void* x_codes, int64_t codes_stride, int split, int pairs, cudaStream_t s) {
  CUtensorMap map_w, map_x, map_s, map_o = {};
  cudaError_t e = encode_codes(&map_w, w, l.N, l.K, l.K, kCols / 2);
  if (e == cudaSuccess) e = encode_codes(&map_x, x_codes, l.T, l.K, codes_stride, kTokRows);
  if (e == cudaSuccess) e = encode_scales(&map_s, l.x_scale, l.T, l.KB, l.x_scale_stride, kTokRows);
  const int64_t row_bytes = l.out_stride * (kFp32 ? 4 : 2);
  ManyArgs a;
  a.l = l;
  // (TMA writes whole 16 bytes, and so past a row's last output where that leaves some of them:
  // such rows are written by lanes, 4096 x 7168 x 4095 in rows of 4096 91 -> 98 us)
  a.by_tma = reinterpret_cast<uintptr_t>(l.out) % 16 == 0 && row_bytes % 16 == 0 && (int64_t)l.N * (kFp32 ? 4 : 2) % 16 == 0;
  if (e == cudaSuccess && a.by_tma) e = encode_rows(&map_o, l.out, kFp32, l.T, l.N, row_bytes, 32);
  if (e != cudaSuccess) return e;
  a.tiles_t = (l.T + 2 * kTokRows - 1) / (2 * kTokRows);
  a.tiles_n = (l.N + kCols - 1) / kCols;
  const int64_t tiles = (int64_t)a.tiles_t * a.tiles_n;
  if (tiles > 1 << 30) return cudaErrorInvalidValue;
  a.tiles = (int)tiles;
  a.split = split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kShare ? 2 * split * tiles : 2 * std::min<int64_t>(tiles, pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Many<kCols>::SmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2 * split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_many_kernel<kCols, kFp32, kShare>, map_w, map_x, map_s, map_o, a);
}

// Clusters of 2 and 4 pairs that a device runs at once.
std::atomic<int> g_room[64][2];

// How the products are cut up: for the fewest cycles, by the turns that the pairs take with
// tiles 256 or 128 outputs wide (755 cycles a block of K, 424), and, where pairs would have
// nothing to do, with two or four of them to a tile (470), whose join takes longer the
// more there are: 300 x 7168 x 576 14.8 -> 9.4 us with four, 500 x 7168 x 1536 15.2 -> 12.4
// with two, 333 x 4000 x 2051 10.9 and 11.1.
struct Cut {
  int cols, split;
  int64_t cycles;
};
Cut cut_of(int T, int N, int KB, int dev, int pairs) {
  const int64_t rows = (T + 2 * kTokRows - 1) / (2 * kTokRows), wide = rows * ((N + 255) / 256), narrow = rows * ((N + 127) / 128);
  Cut best = {256, 1, (wide + pairs - 1) / pairs * KB * 755};
  if (const int64_t c = (narrow + pairs - 1) / pairs * KB * 424; c < best.cycles) best = {128, 1, c};
  for (int split = 2; split <= 4; split *= 2)
    if (const int64_t c = (int64_t)((KB + split - 1) / split) * 470 + (1000 + 60 * narrow) * split; c < best.cycles && KB >= 2 * split && narrow <= g_room[dev][split == 4].load())
      best = {128, split, c};
  return best;
}

template <bool kFp32>
cudaError_t launch_cut(const LinearArgs& l, const void* w, const void* x_codes, int64_t codes_stride, int dev, int sms, cudaStream_t s) {
  const int pairs = sms / 2;
  const Cut c = cut_of(l.T, l.N, l.KB, dev, pairs);
  return c.split > 1     ? launch<128, kFp32, true>(l, w, x_codes, codes_stride, c.split, pairs, s)
         : c.cols == 128 ? launch<128, kFp32, false>(l, w, x_codes, codes_stride, 1, pairs, s)
                         : launch<256, kFp32, false>(l, w, x_codes, codes_stride, 1, pairs, s);
}

template <int kCols, bool kFp32, bool kShare>
cudaError_t configure() {
  // the warps' register shares (setmaxnreg) must fit what the launch gives the
  // CTA, or the growing ones would wait for ever
  cudaFuncAttributes f;
  cudaError_t e = cudaFuncGetAttributes(&f, linear_many_kernel<kCols, kFp32, kShare>);
  if (e == cudaSuccess && f.numRegs * kThreads < kFewRegs * 32 * kFirstEpi + kEpiRegs * 32 * kEpiWarps) e = cudaErrorInvalidConfiguration;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(linear_many_kernel<kCols, kFp32, kShare>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Many<kCols>::SmemBytes);
  return e;
}

}  // namespace

cudaError_t configure_linear_many(int dev) {
  cudaError_t e = configure<256, false, false>();
  if (e == cudaSuccess) e = configure<256, true, false>();
  if (e == cudaSuccess) e = configure<128, false, false>();
  if (e == cudaSuccess) e = configure<128, true, false>();
  if (e == cudaSuccess) e = configure<128, false, true>();
  if (e == cudaSuccess) e = configure<128, true, true>();
  for (int split = 2; split <= 4 && e == cudaSuccess; split *= 2) {
    int n = 0;
    e = active_clusters(linear_many_kernel<128, false, true>, 2 * split, kThreads, Many<128>::SmemBytes, &n);
    g_room[dev][split == 4].store(n);
  }
  return e;
}

int64_t linear_many_cycles(int T, int N, int KB, int dev, int sms) { return cut_of(T, N, KB, dev, sms / 2).cycles; }

cudaError_t launch_linear_many(const LinearArgs& l, const void* w, const void* x_codes, int64_t codes_stride, int dev, int sms, cudaStream_t s) {
  return l.out_fp32 ? launch_cut<true>(l, w, x_codes, codes_stride, dev, sms, s) : launch_cut<false>(l, w, x_codes, codes_stride, dev, sms, s);
}

}  // namespace fw
