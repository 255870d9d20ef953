// Attention for requests that bring many query rows (prompts and chunks of
// them): a dense contraction per (request, key/value head), on the tcgen05
// tensor cores.
//
//   S = Q K^T,  P = 2^(scale S - m),  O = sum over key tiles of P V,  out = O / l
//
// The rows of a head's group are packed (row = new token x G + head in the
// group), so a key/value head's tiles serve all its query heads. A CTA owns
// 256 rows as two 128-row tiles, and walks the 128-key tiles that they see.
// While one row tile is in its softmax the tensor core works on the other: per
// row tile the steps S(i) -> P(i) -> O(i) are serial, S and P share
// tensor-memory columns, and the issue order PV(i), QK(i + 1) of one warp is
// all the ordering that needs.
//
// The 4-bit tiles are unpacked to 16-bit operands (K by keys, V transposed by
// dims, both K-major with the 128-byte swizzle) in one of two places. Where
// many row blocks read each key tile (kReady), a kernel before this one
// unpacks every tile once, into the workspace, as the very bytes of the shared
// memory it will lie in, and one bulk copy brings a tile. Where few do, four
// warps of the CTA unpack its own tiles.
//
// Warps: those of the softmax, row tile 0's first (one or two threads a row: no
// shuffles), then four unpacking warps (not kReady), two that issue the MMAs,
// one that copies tiles or pages. The chain S -> P -> O -> S of a row tile
// bounds it: 1024 cycles of products, about 900 of softmax, and four barriers
// of about 175 from arrival to wake.
//
// Tensor memory: S0 | S1 | O0 | O1, 128 columns each; P (f16) over the first
// 64 columns of its S. Shared memory: Q, a ring of operand tiles taken in the
// order K0 V0 K1 V1 ..., and (not kReady) a ring of packed tiles.
#include <initializer_list>
#include <type_traits>

#include "attn.cuh"
#include "tcgen05.cuh"

namespace fw {
namespace {

using namespace dev;

constexpr int kRowTile = 128, kBlockRows = 2 * kRowTile;
constexpr int kPacked = 3, kHave = 8;
constexpr uint32_t kTmemCols = 512;
// not kReady: registers of the softmax warps and of the others, of 128 a thread at launch
constexpr int kSoftmaxRegs = 184, kOtherRegs = 72;
constexpr float kMost = 32768.f;  // a row's maximum moves only when a tile's sum of p passes this (f16 holds 65504)
// log2 of a row's largest p when its maximum is set. p as f16, good to
// 2^-25 at least, is then good to 2^-28 of the row's largest. (At 8 rows of windowed
// prompts pass kMost more often: 59.9 us instead of 53.0; at 0 51.5.)
constexpr int kTop = 4;

// What goes with an unpacked tile of a head.
struct __align__(16) TileInfo {
  uint32_t have;                // bit g: the keys 16 g .. 16 g + 15 are there
  uint8_t flag[4];              // per 32 keys: some scale of V is not finite
  int32_t wide;                 // values and probabilities in bf16, else in f16
  uint32_t pad;
  float key[4];                 // per 32 keys: the power of two their scales were divided by (kReady: all the same)
  uint8_t poison[kStageKeys];   // then: the key's blocks (bits) that are not
};

template <int D>
struct Cfg {
  static constexpr int NB = D / kKvBlock;
  static constexpr uint32_t QBytes = kRowTile * D * 2;       // one row tile: [D / 64] panels of [128 rows][128 B]
  static constexpr uint32_t TileBytes = kStageKeys * D * 2;  // K: as Q; V: [2] panels of 64 keys, [D dims][128 B]
  static constexpr uint32_t PackedBytes = kStageKeys * D * 9 / 8;
  // an unpacked tile in the workspace: K, V, TileInfo
  static constexpr int64_t ReadyBytes = 2 * TileBytes + 256;
};
static_assert(sizeof(TileInfo) <= 256 && sizeof(TileInfo) % 16 == 0, "TileInfo is copied in bulk");

template <int D, bool kReady>
struct Lay {
  // Threads of a row: with two, a sub-core has two warps of a row tile whose
  // exponentials and other steps overlap (one warp issues in order).
  static constexpr int Split = kReady ? 2 : 1, Cols = kStageKeys / Split, SoftmaxWarps = 8 * Split;
  static constexpr int UnpackWarp0 = SoftmaxWarps, MmaWarp = SoftmaxWarps + (kReady ? 0 : 4), LoadWarp = MmaWarp + 2;
  static constexpr int Threads = kReady ? 608 : 512;
  static constexpr int Tiles = kReady ? 4 : 3;  // ring of operand tiles
  static constexpr uint32_t SmemBytes = 2 * Cfg<D>::QBytes + Tiles * Cfg<D>::TileBytes + (kReady ? 0 : kPacked * Cfg<D>::PackedBytes) + 1024;
};

struct PrefillArgs {
  fw_attn_q4_args u;
  int splits;        // CTAs that share a block's key tiles
  int min_rows;      // requests of at most so many rows are not this kernel's
  int blocks;        // blocks of 256 rows at most (grid = blocks * n_kv * splits)
  uint8_t* ready;    // kReady: [tiles of all requests][n_kv] unpacked tiles
  float* o;          // splits > 1: [blocks * n_kv * splits][256][D]
  float2* ml;        // [blocks * n_kv * splits][256]
  SplitRecord* rec;  // [blocks * n_kv]
  float scale_log2;
};

// Keys and values go to f16: d (c - 8) has at most 8 + 3 significant bits, so
// f16 holds it exactly from 2^-17 of scale to 2^13.
// Keys: what f16 lacks in range is made up by powers of two. A query row is
// divided by its largest magnitude's, and the keys of a tile (kReady, else of 32
// positions: one warp's, which need not wait for the others') by one that brings
// their largest scale to 2^11..2^12; both go back into the factor of the scores. So
// keys are exact unless scales of one tile differ by 2^28 and more, and then good
// to 2^-37 of the largest key, as a row's elements below 2^-14 of its largest are to
// 2^-25 of that.
// Values: a tile whose scales all lie in [2^-10, 2^4) -- blocks with a largest
// magnitude of 2^-7 to 2^7 -- or are zero goes in f16, exactly, and so do its
// probabilities, to 2^-11: the output's own rounding is then all the error there
// is (0.0017 against 64 bits; with bf16 for both 0.0026, and 1 to 4 % of the time
// less). Any other tile goes in bf16, values and probabilities rounded: each tile's
// product has its own type. What size a tile's values have never enters its
// probabilities: f16 has no room for it (kTop) beside the weights themselves, and
// what it drops at the bottom, 2^-28 of a row's largest, is nothing only as long as
// the values it belongs to are not that much larger than the others: at most 2^14
// times, by the window.
constexpr uint32_t kNarrowLow = 127 - 10, kNarrow = 14;  // f16 tiles: lowest exponent of a scale (biased), and how many

// nibbles 2 k + {0, 1} (and + 4) of a word, shifted to the low byte of each
// half -> two f16 pairs (c - 8) d, exact; the upper nibble stands for 16 c as it is
__device__ __forceinline__ void unpack_f16(uint32_t w, uint32_t mask, uint32_t mask4, uint32_t d, uint32_t& lo, uint32_t& hi) {
  uint32_t x, y;
  asm("lop3.b32 %0, %1, %2, 0x64006400, 0xEA;" : "=r"(x) : "r"(w), "r"(mask));        // 1024 + c
  asm("lop3.b32 %0, %1, %2, 0x64006400, 0xEA;" : "=r"(y) : "r"(w), "r"(mask4));   // 1024 + 16 c
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(0x64086408u));               // - 1032
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(y), "r"(0x2C002C00u), "r"(0xD480D480u));  // / 16 - 72
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(d));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(d));
}
__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// nibbles at bit `shift` of a word's halves -> (c - 8) * d, exact in f16 or
// rounded once to bf16
template <bool kHalf>
__device__ __forceinline__ uint32_t unpack(uint32_t w, int shift, uint32_t mask, uint32_t d) {
  uint32_t r;
  if constexpr (kHalf) {
    asm("lop3.b32 %0, %1, %2, 0x64006400, 0xEA;" : "=r"(r) : "r"(w >> shift), "r"(mask));  // 1024 + c
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x64086408u));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(d));
  } else {
    asm("lop3.b32 %0, %1, %2, 0x43004300, 0xEA;" : "=r"(r) : "r"(w >> shift), "r"(mask));  // 128 + c
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x43084308u));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(d));
  }
  return r;
}
__device__ __forceinline__ bool finite_bf16(uint32_t bits) { return (bits & 0x7F80u) != 0x7F80u; }

// A request's tokens and key tiles as far as this kernel takes it.
__device__ __forceinline__ bool prefill_request(const PrefillArgs& a, int r, int& n, int& q0, int& S) {
  const fw_attn_q4_args& u = a.u;
  q0 = u.q_start[r];
  n = u.q_start[r + 1] - q0;
  S = ::min(u.seq_lens[r], u.max_blocks * u.page);
  return sound_queries(u, q0, n) && n * (long long)(u.n_q / u.n_kv) > a.min_rows;
}
__device__ __forceinline__ int key_tiles(int S) { return S > 0 ? (S + kStageKeys - 1) / kStageKeys : 0; }

// 32 keys of a packed tile (a lane a key) -> K operand tile. key0: the tile's
// first key; have: its keys that are there. Only those, up to the request's last,
// decide what the scales are divided by: anything may lie in the others' places.
template <int D, bool kReady>
__device__ __forceinline__ void unpack_keys(uint8_t* tile, const uint8_t* pk, int w, int lane, int page, int page_shift, uint32_t hb,
                                            const KvPlanes& pl, uint32_t mask, int key0, int S, uint32_t have, TileInfo* info) {
  constexpr int NB = Cfg<D>::NB;
  const int key = 32 * w + lane, at = key & (page - 1);
  const uint8_t* blk = pk + (key >> page_shift) * hb;
  const uint8_t* codes = blk + at * (D / 2);
  uint32_t sc[NB / 2], top = 0;
#pragma unroll
  for (int k = 0; k < NB / 2; ++k) {
    sc[k] = reinterpret_cast<const uint32_t*>(blk + pl.ks)[at * (NB / 2) + k];
    const uint32_t even = sc[k] & 0x7FFFu, odd = sc[k] >> 16 & 0x7FFFu;
    top = ::max(top, ::max(even < 0x7F80u ? even : 0u, odd < 0x7F80u ? odd : 0u));
  }
  if (!(have >> (key / 16) & 1) || key0 + key >= S) top = 0;
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if constexpr (kReady) {  // of the tile's four warps
    if (lane == 0) info->key[w] = __uint_as_float(top);
    asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
#pragma unroll
    for (int k = 0; k < 4; ++k) top = ::max(top, __float_as_uint(info->key[k]));
    asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
  }
  // 2^e (any for zeros): between 2^-126 and 2^116
  const int e = top ? ::max((int)(top >> 7) - 127 - 11, -126) : 0;
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
  if (lane == 0) info->key[w] = __uint_as_float((uint32_t)(127 + e) << 23);
  uint32_t d[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const float x = __uint_as_float(b & 1 ? sc[b / 2] & 0xFFFF0000u : sc[b / 2] << 16) * down;
    d[b] = f16x2_bits(x, x);
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
      unpack_f16(x[b], mask, mask << 4, d[b], o.x, o.y);
      unpack_f16(x[b] >> 8, mask, mask << 4, d[b], o.z, o.w);
      *reinterpret_cast<uint4*>(at_q + (b / 2) * (kStageKeys * 128) + (x4 ^ ((b & 1) << 6))) = o;
    }
  }
}

// Barrier of `threads` threads with the OR of their predicates.
__device__ __forceinline__ bool bar_red_or(int id, int threads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)pred)
      : "memory");
  return r != 0;
}

// Whether a packed tile's values need bf16 (see kNarrow): some finite scale, other
// than zero, of the keys that are there is outside of f16's window. This warp's 32
// keys, half a pair's blocks to a lane.
template <int D>
__device__ __forceinline__ bool wide_values(const uint8_t* pk, int w, int lane, int page, int page_shift, uint32_t hb, const KvPlanes& pl,
                                            int key0, int S, uint32_t have) {
  constexpr int NB = Cfg<D>::NB;
  const int kp = 16 * w + lane / 2;
  const uint8_t* at = pk + ((2 * kp) >> page_shift) * hb + pl.vs + (kp & (page / 2 - 1)) * (NB * 4) + (lane & 1) * (NB * 2);
  auto outside = [](uint32_t d) { return d && d < 0x7F80u && (d >> 7) - kNarrowLow >= kNarrow; };
  bool even = false, odd = false;
#pragma unroll
  for (int k = 0; k < NB / 2; ++k) {
    const uint32_t sc = reinterpret_cast<const uint32_t*>(at)[k];
    even |= outside(sc & 0x7FFFu);
    odd |= outside(sc >> 16 & 0x7FFFu);
  }
  return (have >> (kp / 8) & 1) && ((even && key0 + 2 * kp < S) || (odd && key0 + 2 * kp + 1 < S));
}

// 32 keys of a packed tile -> V operand tile, as four 8-key chunks, a lane four
// dims of one block. key0: the tile's first key; have: its keys that are there.
// Scales that must not enter the product -- of keys past the last or of a
// missing page (whatever is there), and what is not finite (noted for the rows
// that see it) -- count as zero.
template <int D>
__device__ __forceinline__ void unpack_values(uint8_t* tile, const uint8_t* pk, int w, int lane, int page, int page_shift, uint32_t hb,
                                              const KvPlanes& pl, uint32_t mask, int key0, int S, uint32_t have, TileInfo* info) {
  constexpr int NB = Cfg<D>::NB;
  const bool wide = info->wide;
  // byte offset of a key pair's codes and scales within the packed tile
  auto codes_at = [&](int kp) { return ((2 * kp) >> page_shift) * hb + pl.vc + (kp & (page / 2 - 1)) * D; };
  auto scales_at = [&](int kp) { return ((2 * kp) >> page_shift) * hb + pl.vs + (kp & (page / 2 - 1)) * (NB * 4); };
  const uint32_t mine = have >> (2 * w) & 3;
  bool odd_tile = mine != 3 || key0 + 32 * w + 32 > S;
  {
    const int kp = 16 * w + lane / 2;  // half a pair's blocks to a lane
    const uint32_t at_s = scales_at(kp);
    uint32_t bad0 = 0, bad1 = 0;       // blocks of the even and the odd key
#pragma unroll
    for (int k = 0; k < NB / 2; ++k) {
      const int b = (lane & 1) * (NB / 2) + k;
      const uint32_t sc = *reinterpret_cast<const uint32_t*>(pk + at_s + b * 4);
      if (!finite_bf16(sc & 0xFFFFu)) bad0 |= 1u << b;
      if (!finite_bf16(sc >> 16)) bad1 |= 1u << b;
    }
    const bool there = mine >> (lane / 16) & 1;
    if (!there || key0 + 2 * kp >= S) bad0 = 0;
    if (!there || key0 + 2 * kp + 1 >= S) bad1 = 0;
    const bool some = __any_sync(0xFFFFFFFFu, (bad0 | bad1) != 0);
    if (some) {
      bad0 |= __shfl_xor_sync(0xFFFFFFFFu, bad0, 1);
      bad1 |= __shfl_xor_sync(0xFFFFFFFFu, bad1, 1);
      if ((lane & 1) == 0) {
        info->poison[2 * kp] = (uint8_t)bad0;
        info->poison[2 * kp + 1] = (uint8_t)bad1;
      }
      odd_tile = true;
    }
    __syncwarp();
    if (lane == 0) info->flag[w] = some;
  }
  constexpr int Lanes = 8 * NB, Chunks = 32 / Lanes;  // lanes of a pair's words; chunks side by side in a warp
  const int word = lane % Lanes, b = word % NB, g = word / NB;
#pragma unroll 1
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
      const bool there = have >> (c / 2) & 1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = key0 + 8 * c + 2 * k;
        if (!there || j >= S || !finite_bf16(d[k] & 0xFFFFu)) d[k] &= 0xFFFF0000u;
        if (!there || j + 1 >= S || !finite_bf16(d[k] >> 16)) d[k] &= 0xFFFFu;
      }
    }
    if (!wide)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        d[k] = f16x2_bits(__uint_as_float(d[k] << 16), __uint_as_float(d[k] & 0xFFFF0000u));
    uint8_t* col = tile + (c / 8) * (D * 128) + (32 * b + 4 * g) * 128;
    const int c4 = (c & 7) ^ ((g & 1) << 2);  // ((dim & 7) = 4 (g & 1) + j)
    auto write = [&](auto half) {
      constexpr bool kHalf = decltype(half)::value;
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int j = (jj + (NB == 4 ? b : 2 * b + (g >> 1))) & 3;  // (the writes of 8 lanes fall into different banks)
        *reinterpret_cast<uint4*>(col + j * 128 + ((c4 ^ j) << 4)) =
            make_uint4(unpack<kHalf>(x[0], 4 * j, mask, d[0]), unpack<kHalf>(x[1], 4 * j, mask, d[1]),
                       unpack<kHalf>(x[2], 4 * j, mask, d[2]), unpack<kHalf>(x[3], 4 * j, mask, d[3]));
      }
    };
    if (wide)
      write(std::false_type{});
    else
      write(std::true_type{});
  }
}

__device__ __forceinline__ uint32_t code_mask() {  // a variable for the compiler: see unpack
  uint32_t m;
  asm volatile("mov.u32 %0, 0x000F000F;" : "=r"(m));
  return m;
}

// The pages of key tile `block` of request r that some row of positions
// first .. last sees, one to a lane (`need`), by bulk copies into `dst`.
// have_out: the tile's keys that come (16 to a bit).
__device__ __forceinline__ void copy_pages(uint8_t* dst, uint64_t* full, const fw_attn_q4_args& u, bool need, int id, int head,
                                               uint32_t hb, int page_shift, int lane, uint32_t* have_out) {
  bool copy = need;
  if (copy && (id < 0 || id >= u.n_pages)) {
    copy = false;
    raise(u.status, FW_KV_BAD_SLOT);
  }
  const uint32_t got = __ballot_sync(0xFFFFFFFFu, copy);
  uint32_t have = 0;  // a page's bit, for each 16 keys of it
#pragma unroll
  for (int k = 0; k < kStageKeys / 16; ++k) have |= (got >> ((k * 16) >> page_shift) & 1) << k;
  if (lane == 0) {
    *have_out = have;
    mbar_arrive_expect_tx(full, (uint32_t)__popc(got) * hb);
  }
  __syncwarp();
  if (copy) bulk_g2s(dst + lane * hb, (const uint8_t*)u.cache + ((int64_t)id * u.n_kv + head) * hb, hb, full);
}

// ------------------------------------------------------------- unpacking ahead
// One CTA per (tile, head): pages in by bulk copies, warps 0-3 unpack K and 4-7
// V, the operand tiles out by bulk copies. Bound by the 16-bit tiles written.
constexpr int kAheadThreads = 256;
template <int D>
struct AheadSmem {
  static constexpr uint32_t Bytes = 2 * Cfg<D>::TileBytes + 256 + Cfg<D>::PackedBytes;
};

template <int D>
__global__ void __launch_bounds__(kAheadThreads) unpack_ahead_kernel(PrefillArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full;
  __shared__ int s_sum[kAheadThreads / 32], s_found[2];
  const fw_attn_q4_args& u = a.u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = blockIdx.x / u.n_kv, head = blockIdx.x % u.n_kv;
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) {
    mbar_init(&full, 1);
    fence_mbar_init();
    s_found[0] = -1;
  }
  // the request that tile number `tile` belongs to
  int base = 0;
  for (int r0 = 0; r0 < u.R && base <= tile; r0 += kAheadThreads) {
    const int r = r0 + tid;
    int n, q0, S, t = 0;
    if (r < u.R && prefill_request(a, r, n, q0, S)) t = key_tiles(S);
    int inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += x;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    int before = base + inc - t;
#pragma unroll
    for (int w = 0; w < kAheadThreads / 32; ++w) {
      if (w < warp) before += s_sum[w];
      base += s_sum[w];
    }
    if (tile >= before && tile < before + t) {
      s_found[0] = r;
      s_found[1] = tile - before;
    }
  }
  __syncthreads();
  const int r = s_found[0], block = s_found[1];
  if (r < 0) return;  // fewer tiles than the host had to allow for
  int n, q0, S;
  prefill_request(a, r, n, q0, S);
  const int first = S - n, lo_key = u.window ? ::max(0, ::max(0, first) + 1 - u.window) : 0, key0 = block * kStageKeys;
  if (key0 + kStageKeys <= lo_key && key0 >= u.sinks) return;  // no row sees it
  const int page_shift = __ffs(u.page) - 1;
  const uint32_t hb = (uint32_t)kv_head_bytes(u.page, D);
  const KvPlanes pl = kv_planes(u.page, D);
  uint8_t* pk = smem + 2 * C::TileBytes + 256;
  TileInfo* info = reinterpret_cast<TileInfo*>(smem + 2 * C::TileBytes);
  if (warp == 0) {
    const int key = key0 + (lane << page_shift);
    // (pages in sight only: behind a window they may be others' by now)
    const bool need = lane < (kStageKeys >> page_shift) && key < S && (key + u.page > lo_key || key < u.sinks);
    const int id = need ? u.block_table[(int64_t)r * u.max_blocks + (key >> page_shift)] : 0;
    copy_pages(pk, &full, u, need, id, head, hb, page_shift, lane, &info->have);
  }
  __syncthreads();
  if (!mbar_wait(&full, 0)) raise(u.status, FW_KV_TIMEOUT);
  const uint32_t mask = code_mask();
  if (warp < 4) {
    unpack_keys<D, true>(smem, pk, warp, lane, u.page, page_shift, hb, pl, mask, key0, S, info->have, info);
  } else {
    info->wide = bar_red_or(1, 128, wide_values<D>(pk, warp - 4, lane, u.page, page_shift, hb, pl, key0, S, info->have));
    __syncwarp();
    unpack_values<D>(smem + C::TileBytes, pk, warp - 4, lane, u.page, page_shift, hb, pl, mask, key0, S, info->have, info);
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    bulk_s2g(a.ready + (int64_t)blockIdx.x * C::ReadyBytes, smem, 2 * C::TileBytes + (uint32_t)sizeof(TileInfo));
    bulk_s2g_wait();
  }
}

// ------------------------------------------------------------- the attention
// A bounded wait with its loop in place (where warps change their register
// share a call would need a register split of its own) and without a suspend
// hint: from arrival to wake 175 cycles instead of 205, four times a tile in the
// chain of softmax and products.
__device__ __forceinline__ bool mbar_wait_inline(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}

// kWindow: with a sliding window nearly all tiles are edges, and what masks
// them has to be cheap; without one only a block's last tiles are, and the
// registers of the other tiles decide.
template <int D, bool kReady, bool kWindow>
__global__ void __launch_bounds__(Lay<D, kReady>::Threads, 1) attn_prefill_kernel(PrefillArgs a) {
  using C = Cfg<D>;
  using Y = Lay<D, kReady>;
  constexpr int kThreads = Y::Threads, kTiles = Y::Tiles;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t packed_full[kPacked], packed_empty[kPacked], tile_full[kTiles], tile_empty[kTiles];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], o_full[2], turn[2], q_full;
  __shared__ TileInfo s_info[kHave];
  __shared__ uint32_t s_tmem;
  __shared__ int s_scan[kThreads / 32], s_scan_tiles[kThreads / 32], s_found[6];
  __shared__ float s_qscale[kBlockRows];  // powers of two the query rows were divided by
  __shared__ float s_pair[2][kBlockRows];  // two threads a row: what they tell each other
  const fw_attn_q4_args& u = a.u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = u.n_q / u.n_kv;
  const int z = blockIdx.x % a.splits, pair = blockIdx.x / a.splits, head = pair % u.n_kv;
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = base;
  uint8_t* sT = sQ + 2 * C::QBytes;
  uint8_t* sP = sT + kTiles * C::TileBytes;  // packed tiles

  if (tid == 0) {
    for (int i = 0; i < kPacked; ++i) {
      mbar_init(&packed_full[i], 1);
      mbar_init(&packed_empty[i], 4);
    }
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&tile_full[i], kReady ? 1 : 4);
      mbar_init(&tile_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&turn[i], 1);
      mbar_init(&p_full[i], 4 * Y::Split);
    }
    mbar_init(&q_full, Y::SoftmaxWarps);
    fence_mbar_init();
  }
  if (warp == Y::MmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  auto tmem_free = [&]() {
    if (warp == Y::MmaWarp)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "r"(kTmemCols) : "memory");
  };
  pdl_wait();
  pdl_launch_dependents();

  // Which block of which request: the blocks in descending order of their
  // place, so that a prompt's later rows, which see the most keys, start first.
  int total = 0, want = -1;
  for (int pass = 0; pass < 2; ++pass) {
    int sum = 0, sum_tiles = 0;
    for (int r0 = 0; r0 < u.R; r0 += kThreads) {
      const int r = r0 + tid;
      int n = 0, q0 = 0, S = 0, nb = 0, nt = 0;
      if (r < u.R && prefill_request(a, r, n, q0, S)) {
        nb = (int)((n * (long long)G + kBlockRows - 1) / kBlockRows);
        nt = key_tiles(S);
      }
      int inc = nb, inc_tiles = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, inc, o), y = kReady ? __shfl_up_sync(0xFFFFFFFFu, inc_tiles, o) : 0;
        if (lane >= o) {
          inc += x;
          inc_tiles += y;
        }
      }
      __syncthreads();
      if (lane == 31) {
        s_scan[warp] = inc;
        s_scan_tiles[warp] = inc_tiles;
      }
      __syncthreads();
      int before = sum + inc - nb, before_tiles = sum_tiles + inc_tiles - nt;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) {
          before += s_scan[w];
          before_tiles += s_scan_tiles[w];
        }
        sum += s_scan[w];
        sum_tiles += s_scan_tiles[w];
      }
      if (pass == 0 && r0 + kThreads >= u.R) {
        total = sum;
        want = total - 1 - pair / u.n_kv;
      }
      // (in the first pass the total, and so the block, is known in the last chunk only)
      if (want >= before && want < before + nb) {
        s_found[0] = r;
        s_found[1] = want - before;
        s_found[2] = n;
        s_found[3] = q0;
        s_found[4] = S;
        s_found[5] = before_tiles;
      }
    }
    if (want < 0 || u.R <= kThreads) break;
  }
  if (want < 0) {  // fewer blocks than the host had to allow for
    if (a.splits > 1 && z == 0 && tid == 0) a.rec[pair].parts = 0;
    tmem_free();
    return;
  }
  __syncthreads();
  const int r = s_found[0], row0 = s_found[1] * kBlockRows, n_new = s_found[2], tok0 = s_found[3];
  const int rows = ::min(kBlockRows, n_new * G - row0), row_tiles = rows > kRowTile ? 2 : 1;
  const int S = s_found[4];
  if (u.seq_lens[r] > S && tid == 0) raise(u.status, FW_KV_BAD_SLOT);  // more positions than the table has pages
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

  if (warp < Y::SoftmaxWarps) {
    // ------------------------------------------------ softmax: one or two threads a row
    if constexpr (!kReady) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    constexpr int Cols = Y::Cols;
    const int t = warp / (4 * Y::Split), half = (warp >> 2) & (Y::Split - 1), row = t * kRowTile + (warp & 3) * 32 + lane;
    // the OR of a predicate over the warps of these 32 rows, which meet it the
    // same number of times whatever happens (after an abandoned wait the loop
    // below runs on without meaning)
    auto any = [&](bool x) {
      if constexpr (Y::Split == 1)
        return __any_sync(0xFFFFFFFFu, x) != 0;
      else
        return bar_red_or(1 + t * 4 + (warp & 3), 64, x);
    };
    // this thread's share of Q into shared memory: 16 bytes a lane, rows of a
    // token side by side (all 256 rows: those past the last are zeros); the
    // loads of a batch all in flight before the first is used
    constexpr int Step = Y::SoftmaxWarps * 32 / (D / 8), Batch = 8;  // rows between a thread's chunks
    static_assert(kBlockRows % Step == 0, "a whole number of rows a pass");
    const int c = tid % (D / 8), step_tok = Step / G, step_head = Step % G;
    int tok = (row0 + tid / (D / 8)) / G, hd = (row0 + tid / (D / 8)) % G;  // of the next row, kept without dividing again
    for (int r0 = tid / (D / 8); r0 < kBlockRows; r0 += Step * Batch) {
      uint4 in[Batch];
#pragma unroll
      for (int k = 0; k < Batch; ++k) {
        in[k] = make_uint4(0, 0, 0, 0);
        if (r0 + k * Step < rows)
          in[k] = *reinterpret_cast<const uint4*>((const __nv_bfloat16*)u.q + (int64_t)(tok0 + tok) * u.q_stride + (head * G + hd) * D + 8 * c);
        tok += step_tok;
        hd += step_head;
        if (hd >= G) {
          hd -= G;
          ++tok;
        }
      }
#pragma unroll
      for (int k = 0; k < Batch; ++k) {
        const int qr = r0 + k * Step;
        if (qr >= kBlockRows) break;
        const uint4 w = in[k];
        float x[8];
        bf16x2_to_f32(w.x, x[0], x[1]);
        bf16x2_to_f32(w.y, x[2], x[3]);
        bf16x2_to_f32(w.z, x[4], x[5]);
        bf16x2_to_f32(w.w, x[6], x[7]);
        // the largest magnitude's exponent: bf16 magnitudes order as their bits
        uint32_t most = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
#pragma unroll
        for (int j = 1; j < D / 8; j <<= 1) most = __vmaxu2(most, __shfl_xor_sync(0xFFFFFFFFu, most, j));
        // 2^e of it, from 2^-100 to 2^126; rows that are not finite as they are
        uint32_t ex = ::max(most << 16, most & 0xFFFF0000u) & 0x7F800000u;
        ex = ex == 0x7F800000u ? 127u << 23 : ::min(::max(ex, 27u << 23), 253u << 23);
        const float down = __uint_as_float((254u << 23) - ex);
        if (c == 0) s_qscale[qr] = __uint_as_float(ex);
        const int rr = qr % kRowTile;
        *reinterpret_cast<uint4*>(sQ + (qr / kRowTile) * C::QBytes + (c / 8) * (kRowTile * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) =
            make_uint4(f16x2_bits(x[0] * down, x[1] * down), f16x2_bits(x[2] * down, x[3] * down),
                       f16x2_bits(x[4] * down, x[5] * down), f16x2_bits(x[6] * down, x[7] * down));
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full);
    if (t < row_tiles) {
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_cols = tmem + lanes + t * 128, o_cols = tmem + lanes + 256 + t * 128;
      const int p = row < rows ? S - n_new + (row0 + row) / G : -1;
      float mz = 0.f, l = 0.f, q_scale = 0.f;
      bool unset = true;  // no maximum yet
      uint32_t poison = 0;
      int key_before = 0;
      // blocks of V that are not finite in keys this row sees (the tile whose product is in O by now)
      auto check_poison = [&](int i, int key0) {
        const TileInfo& info = s_info[i % kHave];
        const uint32_t flags = *reinterpret_cast<const volatile uint32_t*>(info.flag);
        if (flags == 0) return;
        for (int c = 0; c < kStageKeys; ++c)
          if ((flags >> (8 * (c / 32)) & 1) && sees(p, key0 + c, u.window, u.sinks)) poison |= info.poison[c];
      };
      for (int i = 0; i < n_t; ++i) {
        const int key0 = v.block(i0 + i) * kStageKeys;
        const bool edge = key0 + kStageKeys - 1 > first || (kWindow && key0 < last + 1 - u.window);
        wait(&s_full[t], i & 1);
        tc_fence_after();
        // (the first score tells that every row of Q and its scale were written)
        if (i == 0) q_scale = s_qscale[row];
        // what the scores' products stand for, for each 32 keys (kReady: for all);
        // never zero or infinite, so that -inf and 0 stay what they are
        auto factor = [&](int g) { return fminf(fmaxf(a.scale_log2 * s_info[i % kHave].key[g] * q_scale, 1e-37f), 1e38f); };
        constexpr int Groups = kReady ? 1 : Cols / 32;
        float scale[Groups];
#pragma unroll
        for (int g = 0; g < Groups; ++g) scale[g] = factor(g);
        const uint32_t have = s_info[i % kHave].have >> (half * (Cols / 16));
        const bool masks = edge || (have & ((1u << (Cols / 16)) - 1)) != (1u << (Cols / 16)) - 1;
        // A tile's scores to its P, in f16 or in bf16. The whole of it is there
        // twice: with the two conversions beside each other in the inner loop
        // three chunks took 413 us instead of 327.
        auto tile = [&](auto narrow) {
          // P against the maximum as last set. P and O are exact to their
          // rounding whatever their magnitude, so the maximum only moves (by
          // whole powers of two) when a tile's sum shows that some p is past
          // kMost, or when none was set yet; it is not even taken otherwise.
          // a new maximum from this thread's largest score, in log2
          auto move = [&](float up) {
            if constexpr (Y::Split == 2) {
              s_pair[half][row] = up;
              any(false);
              up = fmaxf(up, s_pair[half ^ 1][row]);
            }
            up = ceilf(up - mz) - kTop;
            // a first maximum is taken as it is, a later one only moves up
            if (!unset) up = fmaxf(up, 0.f);
            const bool moves = up != -INFINITY;
            const float keep = unset ? 0.f : exp2_fast(-up);
            if (moves) {
              mz += up;
              l *= keep;
              unset = false;
            }
            if (i > 0)  // O holds the tiles before: S(i) came after their product
#pragma unroll 1
              for (int c = half * (D / Y::Split); c < (half + 1) * (D / Y::Split); c += 8) {  // 8 columns at a time: S holds the registers
                uint32_t w[8];
                tmem_ld(o_cols + c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (moves) w[j] = __float_as_uint(__uint_as_float(w[j]) * keep);
                tmem_st8(o_cols + c, w);
              }
          };
          uint32_t pk[Cols / 32][16];
          // p of scores, into pk from column c0 on, and their sum
          auto exps = [&](auto& s, int c0) {
            constexpr int N = sizeof(s) / 8;
            const f2 mm = f2_pack(-mz, -mz);
            f2 sums[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < N; ++c) {
              float x, y;
              const float k = scale[(c0 / 32 + c / 16) % Groups];
              f2_unpack(f2_fma(f2_pack_bits(s[2 * c], s[2 * c + 1]), f2_pack(k, k), mm), x, y);
              x = exp2_fast(x);
              y = exp2_fast(y);
              sums[c & 1] = f2_add(sums[c & 1], f2_pack(x, y));
              pk[(c0 / 2 + c) / 16][c % 16] = decltype(narrow)::value ? f16x2_bits(x, y) : bf16x2_bits(x, y);
            }
            float x, y;
            f2_unpack(f2_add(sums[0], sums[1]), x, y);
            return x + y;
          };
          auto largest = [](auto& s, int c0) {  // of 32 columns
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; ++c) top[c & 3] = fmaxf(top[c & 3], __uint_as_float(s[c0 + c]));
            return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          };
          float sum;
          for (int pass = 0;; ++pass) {
            if constexpr (!kWindow) {
              uint32_t s[Cols];
              tmem_ld(s_cols + half * Cols, s);
              if (masks) {
                // (the full condition, although there is no window: the compiler
                // makes worse code of the shorter one, three chunks 461 us instead of
                // 331, and of words of bits as below 338)
                const int at = key0 + half * Cols, hi = p - at, lo = u.window ? hi - u.window : -1, sk = u.sinks - at;
#pragma unroll
                for (int c = 0; c < Cols; ++c)
                  if (!(c <= hi && (c > lo || c < sk) && (have >> (c / 16) & 1))) s[c] = 0xFF800000u;  // -inf
              }
              if (pass == 1 || i == 0) {
                float up = -INFINITY;
#pragma unroll
                for (int w = 0; w < Cols / 32; ++w) up = fmaxf(up, largest(s, 32 * w) * scale[w % Groups]);
                move(up);
              }
              sum = exps(s, 0);
            } else {
              // 32 columns at a time; what a row sees of them (c <= hi, and c > lo
              // or c < sk) as a word of bits: a test and a select each (three
              // comparisons each: windowed prompts took 67 us instead of 55)
              auto scores = [&](auto masked, uint32_t(&s)[32], int w) {
                tmem_ld(s_cols + half * Cols + 32 * w, s);
                if constexpr (decltype(masked)::value) {
                  const int at = key0 + half * Cols + 32 * w, hi = p - at, lo = hi - u.window, sk = u.sinks - at;
                  auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
                  const uint32_t there = (have >> (2 * w) & 1 ? 0xFFFFu : 0u) | (have >> (2 * w + 1) & 1 ? 0xFFFF0000u : 0u);
                  const uint32_t m = below(hi + 1) & (~below(lo + 1) | below(sk)) & there;
#pragma unroll
                  for (int c = 0; c < 32; ++c)
                    if (!(m >> c & 1)) s[c] = 0xFF800000u;
                }
              };
              if (pass == 1 || i == 0) {
                float up = -INFINITY;
#pragma unroll 1
                for (int w = 0; w < Cols / 32; ++w) {
                  uint32_t s[32];
                  scores(std::true_type{}, s, w);
                  up = fmaxf(up, largest(s, 0) * factor(kReady ? 0 : w));
                }
                move(up);
              }
              auto all = [&](auto masked) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < Cols / 32; ++w) {
                  uint32_t s[32];
                  scores(masked, s, w);
                  sum += exps(s, 32 * w);
                }
                return sum;
              };
              sum = masks ? all(std::true_type{}) : all(std::false_type{});
            }
            // (P will lie over S: by now all warps of these rows have read it)
            if (!any(pass == 0 && (unset || sum > kMost))) break;
          }
          l += sum;
#pragma unroll
          for (int c = 0; c < Cols / 32; ++c) tmem_st16(s_cols + half * (Cols / 2) + 16 * c, pk[c]);
        };
        if (__builtin_expect(s_info[i % kHave].wide, 0))
          tile(std::false_type{});
        else
          tile(std::true_type{});
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
        // (S(i) told that tile i - 1 had been unpacked; its notes stay until this row tile's next P)
        if (i > 0) check_poison(i - 1, key_before);
        key_before = key0;
      }
      // ---------------------------------------------- out = O / l
      if constexpr (Y::Split == 2) {
        any(false);  // (s_pair may still be read)
        s_pair[half][row] = l;
        any(false);
        l = s_pair[0][row] + s_pair[1][row];
      }
      if (n_t > 0) {
        wait(&o_full[t], 0);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok) check_poison(n_t - 1, key_before);
      }
      const int n = row0 + row;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (a.splits > 1 && half == 0 && row < rows) a.ml[part * kBlockRows + row] = make_float2(unset ? -INFINITY : mz, l);
#pragma unroll 1
      for (int c = half * (D / Y::Split); c < (half + 1) * (D / Y::Split); c += 32) {
        uint32_t o[32];
        if (n_t > 0 && ok) {
          tmem_ld(o_cols + c, o);
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
  } else if (warp < Y::MmaWarp) {
    // ------------------------------------------------ unpack 4-bit codes to operand tiles
    if constexpr (!kReady) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      const int w = warp - Y::UnpackWarp0;
      const uint32_t mask = code_mask();
      for (int i = 0; i < n_t; ++i) {
        const uint8_t* pk = sP + (i % kPacked) * C::PackedBytes;
        TileInfo* info = &s_info[i % kHave];
        const int key0 = v.block(i0 + i) * kStageKeys;
        wait(&packed_full[i % kPacked], (i / kPacked) & 1);
        // the tile's type, of all four warps; these meet as often as there are
        // tiles, whatever happens (after an abandoned wait without meaning)
        const bool wide = bar_red_or(1, 128, ok && wide_values<D>(pk, w, lane, u.page, page_shift, hb, pl, key0, S, info->have));
        uint32_t seq = 2 * i;
        wait(&tile_empty[seq % kTiles], ((seq / kTiles) & 1) ^ 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) continue;
        info->wide = wide;
        unpack_keys<D, false>(sT + (seq % kTiles) * C::TileBytes, pk, w, lane, u.page, page_shift, hb, pl, mask, key0, S, info->have, info);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tile_full[seq % kTiles]);
        seq = 2 * i + 1;
        wait(&tile_empty[seq % kTiles], ((seq / kTiles) & 1) ^ 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) continue;
        unpack_values<D>(sT + (seq % kTiles) * C::TileBytes, pk, w, lane, u.page, page_shift, hb, pl, mask, key0, S, info->have, info);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&tile_full[seq % kTiles]);
          mbar_arrive(&packed_empty[i % kPacked]);
        }
      }
    }
  } else {
    if constexpr (!kReady) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < Y::MmaWarp + row_tiles) {
      // ---------------------------------------------- MMA issuers, one for each row tile
      // A warp stays together and elects a lane for the MMAs only: their
      // descriptors are then uniform. What an issuer has to wait for and work
      // out takes some hundred cycles a tile, which the other's products hide.
      // The batches PV(i), QK(i + 1) go strictly in turn: left to themselves
      // the two row tiles fall into step, and softmax and products would take
      // turns instead of overlapping.
      const int t = warp - Y::MmaWarp;
      // (a value shuffled from lane 0 is uniform for the compiler, too)
      const uint32_t q0 = __shfl_sync(0xFFFFFFFFu, sw128_desc_lo(smem_u32(sQ) + t * C::QBytes), 0);
      const uint32_t t0 = __shfl_sync(0xFFFFFFFFu, sw128_desc_lo(smem_u32(sT)), 0);
      const uint32_t s_cols = __shfl_sync(0xFFFFFFFFu, tmem + t * 128, 0), o_cols = __shfl_sync(0xFFFFFFFFu, tmem + 256 + t * 128, 0);
      auto ready = [&](uint64_t* bar, uint32_t parity) {
        wait(bar, parity);
        return ok = __all_sync(0xFFFFFFFFu, ok);
      };
      auto tile_ready = [&](uint32_t seq) { return ready(&tile_full[seq % kTiles], (seq / kTiles) & 1); };
      bool go = n_t > 0 && ready(&q_full, 0);
      for (int i = -1; i < n_t && go; ++i) {  // the batch PV(i), QK(i + 1)
        const bool first_batch = i < 0, next = i + 1 < n_t;
        const uint32_t sv = 2 * i + 1, sk = 2 * i + 2;
        if ((!first_batch && !tile_ready(sv)) || (next && !tile_ready(sk))) break;
        if (row_tiles == 2 && !(t == 0 && first_batch) && !ready(&turn[t], (i + t) & 1)) break;
        const uint32_t idesc_v = !first_batch && s_info[i % kHave].wide ? idesc_bf16(kRowTile, D) : idesc_f16(kRowTile, D);
        if (!first_batch && !ready(&p_full[t], i & 1)) break;  // (what comes last is what the chain waits for)
        tc_fence_after();
        if (elect_one()) {
          if (!first_batch) {
            const uint32_t v0 = t0 + (sv % kTiles) * (C::TileBytes >> 4);
#pragma unroll
            for (int k = 0; k < kStageKeys / 16; ++k)
              mma_ts_lo(o_cols, s_cols + k * 8, v0 + (((k / 4) * (D * 128) + (k % 4) * 32) >> 4), idesc_v, i > 0 || k != 0);
            mma_commit(&tile_empty[sv % kTiles]);
            if (row_tiles == 1) mma_commit(&tile_empty[sv % kTiles]);  // (the barrier counts both issuers)
          }
          if (next) {
            const uint32_t k0 = t0 + (sk % kTiles) * (C::TileBytes >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {  // (both tiles have 128 rows)
              const uint32_t at = ((k / 4) * (kRowTile * 128) + (k % 4) * 32) >> 4;
              mma_ss_lo(s_cols, q0 + at, k0 + at, idesc_f16(kRowTile, kStageKeys), k != 0);
            }
            mma_commit(&s_full[t]);
            mma_commit(&tile_empty[sk % kTiles]);
            if (row_tiles == 1) mma_commit(&tile_empty[sk % kTiles]);
          }
          if (row_tiles == 2) mbar_arrive(&turn[t ^ 1]);
        }
        __syncwarp();
      }
      // every MMA issued has finished before tensor memory is read or released
      if (go) {
        if (elect_one()) mma_commit(&o_full[t]);
        __syncwarp();
        mbar_wait_inline(&o_full[t], 0);
      }
    } else if (warp == Y::LoadWarp) {
      int issued = 0;  // tiles whose copies were started
      if constexpr (kReady) {
        // -------------------------------------------- unpacked tiles
        const uint8_t* src = a.ready + (int64_t)s_found[5] * u.n_kv * C::ReadyBytes;
        for (int seq = 0; seq < 2 * n_t; ++seq) {
          const int i = seq / 2, slot = seq % kTiles;
          wait(&tile_empty[slot], ((seq / kTiles) & 1) ^ 1);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          if (elect_one()) {
            const uint8_t* tile = src + ((int64_t)v.block(i0 + i) * u.n_kv + head) * C::ReadyBytes;
            mbar_arrive_expect_tx(&tile_full[slot], C::TileBytes + (seq & 1 ? 0 : (uint32_t)sizeof(TileInfo)));
            bulk_g2s(sT + slot * C::TileBytes, tile + (seq & 1) * C::TileBytes, C::TileBytes, &tile_full[slot]);
            if (!(seq & 1)) bulk_g2s(&s_info[i % kHave], tile + 2 * C::TileBytes, sizeof(TileInfo), &tile_full[slot]);
          }
          __syncwarp();
          issued = seq + 1;
        }
        // copies still in flight after an abandoned wait land before the CTA leaves
        if (!ok)
          for (int j = ::max(0, issued - kTiles); j < issued; ++j) mbar_wait_inline(&tile_full[j % kTiles], (j / kTiles) & 1);
      } else {
        // -------------------------------------------- pages, one to a lane
        int id = 0;
        auto look = [&](int i) {
          const int key = v.block(i0 + i) * kStageKeys + (lane << page_shift);
          const bool need = lane < (kStageKeys >> page_shift) && key <= last && (key + u.page > lo_key || key < u.sinks);
          if (need) id = u.block_table[(int64_t)r * u.max_blocks + (key >> page_shift)];
          return need;
        };
        bool need = n_t > 0 && look(0);
        for (int i = 0; i < n_t; ++i) {
          const bool copy = need;
          const int page = id, slot = i % kPacked;
          if (i + 1 < n_t) need = look(i + 1);  // in flight during this tile
          wait(&packed_empty[slot], ((i / kPacked) & 1) ^ 1);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          // (what the tile has is written before the arrival that lets others read it)
          copy_pages(sP + slot * C::PackedBytes, &packed_full[slot], u, copy, page, head, hb, page_shift, lane, &s_info[i % kHave].have);
          issued = i + 1;
        }
        if (!ok)
          for (int j = ::max(0, issued - kPacked); j < issued; ++j) mbar_wait_inline(&packed_full[j % kPacked], (j / kPacked) & 1);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  tmem_free();
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

// Key tiles of all requests at most.
int64_t most_tiles(const fw_attn_q4_args& a) {
  return (int64_t)a.R * (((int64_t)a.max_blocks * a.page + kStageKeys - 1) / kStageKeys);
}
int64_t ready_bytes(const fw_attn_q4_args& a) {
  return most_tiles(a) * a.n_kv * (a.D == 64 ? Cfg<64>::ReadyBytes : Cfg<128>::ReadyBytes);
}

// Whether tiles are unpacked ahead: where a request has kReadyBlocks row blocks
// or more to read them (on average), and the workspace for all that the block
// tables can hold stays moderate. Eight requests with 4,000 cached positions
// and 32 query heads over 4: at 8 blocks 140 us ahead, 162 us in the kernel; at 6
// 137 and 158, at 4 80 and 82; at 2 blocks (16 requests, 8,000 positions) 177 and 143.
constexpr int kReadyBlocks = 6;
constexpr int64_t kReadyMost = 1ll << 30;
bool prefill_ready(const fw_attn_q4_args& a, int sms) {
  return prefill_splits(a, sms) == 1 && (int64_t)a.T * (a.n_q / a.n_kv) >= (int64_t)kReadyBlocks * kBlockRows * a.R &&
         ready_bytes(a) <= kReadyMost;
}

template <int D, bool kReady, bool kWindow>
cudaError_t configure() {
  using Y = Lay<D, kReady>;
  const auto kernel = attn_prefill_kernel<D, kReady, kWindow>;
  if (!kReady) {
    // the warps' register shares (setmaxnreg) must fit what the launch gives
    // the CTA, or the growing ones would wait for ever
    cudaFuncAttributes f;
    const cudaError_t e = cudaFuncGetAttributes(&f, kernel);
    if (e != cudaSuccess) return e;
    if (f.numRegs * Y::Threads < kSoftmaxRegs * 256 + kOtherRegs * (Y::Threads - 256)) return cudaErrorInvalidDeviceFunction;
  }
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Y::SmemBytes);
}
template <int D>
cudaError_t configure() {
  for (const cudaError_t e : {configure<D, false, false>(), configure<D, false, true>(), configure<D, true, false>(), configure<D, true, true>()})
    if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(unpack_ahead_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, AheadSmem<D>::Bytes);
}

template <int D, bool kReady>
cudaError_t launch_attention(const PrefillArgs& d, int64_t ctas, cudaStream_t s) {
  using Y = Lay<D, kReady>;
  return launch_dependent(d.u.window ? attn_prefill_kernel<D, kReady, true> : attn_prefill_kernel<D, kReady, false>, dim3((unsigned)ctas),
                          dim3(Y::Threads), Y::SmemBytes, s, d);
}
template <int D>
cudaError_t launch(const PrefillArgs& d, int64_t ctas, cudaStream_t s) {
  if (!d.ready) return launch_attention<D, false>(d, ctas, s);
  const int64_t tiles = most_tiles(d.u) * d.u.n_kv;
  const cudaError_t e = launch_dependent(unpack_ahead_kernel<D>, dim3((unsigned)tiles), dim3(kAheadThreads), AheadSmem<D>::Bytes, s, d);
  return e == cudaSuccess ? launch_attention<D, true>(d, ctas, s) : e;
}

}  // namespace

cudaError_t configure_prefill_attn() {
  const cudaError_t e = configure<64>();
  return e == cudaSuccess ? configure<128>() : e;
}

int64_t prefill_workspace(const fw_attn_q4_args& a, int sms) {
  if (prefill_ready(a, sms)) return ready_bytes(a);
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
  d.ready = prefill_ready(a, sms) ? static_cast<uint8_t*>(workspace) : nullptr;
  d.rec = static_cast<SplitRecord*>(workspace);
  d.o = reinterpret_cast<float*>(d.rec + pairs);
  d.ml = reinterpret_cast<float2*>(d.o + pairs * d.splits * kBlockRows * a.D);
  d.scale_log2 = a.scale * kLog2e;
  cudaError_t e = a.D == 64 ? launch<64>(d, pairs * d.splits, s) : launch<128>(d, pairs * d.splits, s);
  if (e == cudaSuccess && d.splits > 1) e = launch_attn_join(a, d.rec, d.o, d.ml, (int)pairs, kBlockRows, s);
  return e;
}

}  // namespace fw
