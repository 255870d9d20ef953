// Attention for requests that bring few query rows (new tokens x heads that
// share a key/value head, at most 16): single tokens and short drafts over
// long contexts. Every key and value is used by few rows: what the kernel cannot
// do without is streaming the 4-bit cache from HBM. What bounds it is latency, with
// 16 warps an SM (128 registers a thread) and some 330 instructions for 16 keys:
// half of the issue slots, 42 to 54 % of HBM and a third of the tensor pipe are busy,
// and warps wait for the results of their own instructions most.
//
//   s[t, n] = sum_b d_k[t, b] sum_{i in b} q[n, i] (c[t, i] - 8)
//   o[n, i] = sum_t (p[t, n] d_v[t, b(i)]) (c'[t, i] - 8)
//
// The block scales are taken out of the products: what enters the tensor
// cores as their 16-row operand are the bare codes (keys in rows for s, dims in
// rows for o), and the query rows are the 8-column operand, so a group of up to
// 8 rows wastes nothing. The codes need no conversion: bf16's smallest numbers
// count up linearly from zero (the subnormals, then the lowest binade), so the
// bits of a whole number c < 256 ARE the bf16 number c 2^-133. A nibble of a
// word's halves is c 2^-133 or, four bits up, 16 c 2^-133: one AND for two of
// them, and one shift for the other four. The other operand makes up for it: the queries are
// multiplied by 2^64 (or 2^60), the probabilities carry 2^64.
// What the codes are too large by (8) is taken back by products as well: for
// the keys one 16-step product of the scales with -8 sum q (in three bf16
// parts), for the values one with the constant -8 in the codes' place -- in the
// same accumulators right after, so that nothing grows before it cancels. p d_v
// is rounded to bf16 once, from p in two bf16 parts: relative error 0.0021 to 0.0023
// against 64 bits where the output's rounding alone gives 0.0017 (p rounded too
// 0.0025 to 0.0028 and 2 to 3 % of the time less; p d_v in two parts as well 0.0017, but
// twice the values' products: single tokens over 98,000-131,000 keys 80 us
// instead of 68).
// (e4m3, whose smallest numbers do the same for bytes, needs fewer operations
// on paper; but this GPU turns 8-bit mma.sync operands into f16 by further
// instructions: 446 instead of 343 of them for 16 keys when both were there.)
//
// Work: a unit is 128 keys of one (request, key/value head); the CTAs take
// consecutive shares of all units, so that ragged lengths and few requests both
// fill the GPU. The shares are equal in cost: a pair costs its units and
// kPairCost more for its query rows, its empty pipeline and its join (64
// requests of 100 to 8191 keys: 77 us at 0, 60 at 3, 52.7 at 6, 52.1 at 8, 53.3 at
// 10; 48 drafts over a window 30.1, 27.9, 26.6, 26.7, 26.9; 4 long contexts 71.6,
// 69.6, 67.8, 67.3, 68.0).
// A unit's pages come into a shared-memory ring by one bulk copy each, which
// the CTA's eight warps issue in turn. Four of them take a unit, 32 keys each,
// the other four the next; each has a softmax state of its own that is joined
// at the end of a segment. A pair whose units fall into several CTAs leaves
// partial results that a second small kernel joins. (Eight warps and no ninth
// as producer: two CTAs of eight leave each warp 128 registers, of nine 96.)
#include <type_traits>

#include "attn.cuh"

namespace fw {
namespace {

using namespace dev;

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kTeam = 4;          // warps of a stage (32 keys each); two teams take the stages in turn
constexpr int kChunk = kThreads;  // requests scanned at a time
constexpr int kPairCost = 6;      // units that a pair costs beside its own: see the work's shares above
constexpr float kLazy = 8.f;      // a row's maximum moves only when a score passes it by 2^8
constexpr float kShift = 64.f;    // probabilities carry 2^64
constexpr float kOScale = 590295810358705651712.f, kLScale = 1.f / 18446744073709551616.f;  // 2^69 = 2^(133 - 64), 2^-64
constexpr uint32_t kLeast = (127 - 48) << 7;  // 2^-48 in bf16
constexpr uint32_t kQUp = 0x5F805F80u, kQUp16 = 0x5D805D80u;  // bf16 pairs of 2^64, 2^60

template <int D, int NT>
struct Cfg {
  static constexpr int NB = D / kKvBlock, Rows = 8 * NT;
  static constexpr int Halves = NT == 1 ? 2 : 1;  // of a warp's 32 keys that are in registers together
  static constexpr uint32_t StageBytes = kStageKeys * D * 9 / 8;
  static constexpr int Stages = D == 128 ? 4 : 8;  // even: a slot is always the same team's
  static_assert(Stages % 2 == 0 && Stages <= kWarps, "see the ring");
  static constexpr int Pitch = D + 4;  // floats between rows of the join buffer: its 16-byte accesses meet no bank twice
  static constexpr uint32_t JoinBytes = kWarps / 2 * 8 * Pitch * 4;
  static constexpr uint32_t QBytes = NT == 1 ? 0 : Rows * D * 2;
  static constexpr uint32_t SmemBytes = Stages * StageBytes + JoinBytes + QBytes;
};

struct DecodeArgs {
  fw_attn_q4_args u;
  float* o;             // [2 grid][Rows][D]
  float2* ml;           // [2 grid][Rows] maximum (log2), sum
  SplitRecord* rec;     // [grid]
  float scale_log2;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t x, uint32_t y, uint32_t z) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void add_release(uint32_t* p) {
  asm volatile("red.release.cta.shared::cta.add.u32 [%0], 1;" ::"r"(smem_u32(p)) : "memory");
}
__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t r;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(r) : "r"(smem_u32(p)) : "memory");
  return r;
}
// Bounded wait for a count to reach n. false = gave up.
__device__ __forceinline__ bool wait_count(const uint32_t* p, uint32_t n) {
  if ((int)(load_acquire(p) - n) >= 0) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if ((int)(load_acquire(p) - n) >= 0) return true;
    if ((i & 63u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}

template <int N>
struct Words {
  uint32_t w[N];
};
template <int N, int Offset>
__device__ __forceinline__ Words<N> lds(uint32_t p) {
  Words<N> r;
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4+%5];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(p), "n"(Offset) : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2+%3];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(p), "n"(Offset) : "memory");
  else
    asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(r.w[0]) : "r"(p), "n"(Offset) : "memory");
  return r;
}

// A segment of a head's keys, for what follows.
struct Segment {
  const uint8_t* cache;   // page 0's block of the head
  const int32_t* pages;   // the request's
  const __nv_bfloat16* q; // the row
  Stages v;
  int st0, n_here, S, p;  // its stages; positions of the request and of the row
};

// Whether some value of a segment's keys is not zero, by the D / 4 lanes of a row.
template <int D>
__device__ __noinline__ bool has_values(const fw_attn_q4_args& u, const Segment& g, int lane4, uint32_t group) {
  constexpr int NB = D / kKvBlock;
  const KvPlanes pl = kv_planes(u.page, D);
  const int page_shift = __ffs(u.page) - 1;
  const int64_t stride = u.n_kv * kv_head_bytes(u.page, D);
#pragma unroll 1
  for (int i = 0; i < g.n_here; ++i) {
    const int key0 = g.v.block(g.st0 + i) * kStageKeys;
    uint32_t bits = 0;
#pragma unroll
    for (int kp = lane4; kp < kStageKeys / 2; kp += D / 4) {
      const int j = key0 + 2 * kp, id = j < g.S ? g.pages[j >> page_shift] : -1;
      if (id < 0 || id >= u.n_pages) continue;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        bits |= reinterpret_cast<const uint32_t*>(g.cache + id * stride + pl.vs)[(j & (u.page - 1)) / 2 * NB + b];
    }
    if (__any_sync(group, (bits & 0x7FFF7FFFu) != 0)) return true;
  }
  return false;
}

// A segment's result for a row from the definition, a key at a time, by its D / 4
// lanes: the mean of the values (this lane's four dims) -> log2 of the sum of
// 2^score (-inf: no key).
template <int D>
__device__ __noinline__ float plainly(const fw_attn_q4_args& u, const Segment& g, int lane4, uint32_t group, float4& mean) {
  constexpr int NB = D / kKvBlock;
  const KvPlanes pl = kv_planes(u.page, D);
  const int page_shift = __ffs(u.page) - 1, b = lane4 / 8, in = lane4 % 8;
  const int64_t stride = u.n_kv * kv_head_bytes(u.page, D);
  const uint2 qw = *reinterpret_cast<const uint2*>(g.q + 4 * lane4);
  float q4[4], o4[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  bf16x2_to_f32(qw.x, q4[0], q4[1]);
  bf16x2_to_f32(qw.y, q4[2], q4[3]);
#pragma unroll 1
  for (int i = 0; i < g.n_here; ++i) {
    const int key0 = g.v.block(g.st0 + i) * kStageKeys, end = ::min(key0 + kStageKeys, g.S);
#pragma unroll 1
    for (int j = key0; j < end; ++j) {
      if (!sees(g.p, j, u.window, u.sinks)) continue;
      const int id = g.pages[j >> page_shift], at = j & (u.page - 1);
      if (id < 0 || id >= u.n_pages) continue;
      const uint8_t* blk = g.cache + id * stride;
      const uint32_t kw = reinterpret_cast<const uint32_t*>(blk + at * (D / 2))[in / 2 * NB + b];
      const uint32_t vw = reinterpret_cast<const uint32_t*>(blk + pl.vc + at / 2 * D)[in * NB + b] >> (16 * (at & 1));
      const float dk = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(blk + pl.ks)[at * NB + b]);
      const float dv = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(blk + pl.vs)[2 * (at / 2 * NB + b) + (at & 1)]);
      float sc = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dim = 4 * (in & 1) + e, nibble = dim / 2 + 4 * (dim % 2);
        sc = fmaf(q4[e], (float)((int)(kw >> (4 * nibble) & 15) - 8), sc);
      }
      sc *= dk;
#pragma unroll
      for (int d = 1; d < D / 4; d <<= 1) sc += __shfl_xor_sync(group, sc, d);
      sc *= u.scale * kLog2e;
      const float up = fmaxf(m, sc), x = exp2_fast(sc - up);
      l = (m == -INFINITY ? 0.f : l * exp2_fast(m - up)) + x;
      m = up;
      const float w = x / l;
#pragma unroll
      for (int e = 0; e < 4; ++e) o4[e] += w * ((float)((int)(vw >> (4 * e) & 15) - 8) * dv - o4[e]);
    }
  }
  mean = make_float4(o4[0], o4[1], o4[2], o4[3]);
  return m == -INFINITY ? m : m + log2f(l);
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2) attn_decode_kernel(DecodeArgs a) {
  using C = Cfg<D, NT>;
  constexpr int NB = C::NB, kStages = C::Stages, H = C::Halves;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kStages];
  __shared__ uint32_t s_left[kStages];       // how often a warp has left the slot
  __shared__ uint32_t s_have[kStages];       // bit w: the stage's keys 16 w .. 16 w + 15 are there
  __shared__ int s_pref[kChunk + 1];         // units before each request of the chunk, from this CTA's first one on
  __shared__ int s_len[kChunk], s_new[kChunk], s_tok[kChunk];
  __shared__ long long s_scan[kWarps][2], s_bound[2];
  __shared__ float2 s_ml[kWarps][C::Rows];
  __shared__ float s_qz[C::Rows][NB];        // -8 x a row's sums over the blocks, in units of the products
  float* join = reinterpret_cast<float*>(smem + kStages * C::StageBytes);
  uint8_t* s_q = smem + kStages * C::StageBytes + C::JoinBytes;  // several row tiles: their query rows
  const fw_attn_q4_args& u = a.u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int G = u.n_q / u.n_kv;
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      s_left[i] = 0;
    }
    fence_mbar_init();
    a.rec[blockIdx.x].parts = 0;
  }

  // a request's units; 0 when it has no rows or more than this kernel takes
  auto request = [&](int r, int& S, int& n, int& q0) -> long long {
    if (r >= u.R) return 0;
    q0 = u.q_start[r];
    n = u.q_start[r + 1] - q0;
    S = u.seq_lens[r];
    if (!sound_queries(u, q0, n) || n < 1 || n * (long long)G > kDecodeRows) return 0;
    if (S > u.max_blocks * u.page) {
      S = u.max_blocks * u.page;
      raise(u.status, FW_KV_BAD_SLOT);
    }
    // an empty context is one unit without keys: its rows are zeros
    return (long long)::max(1, visible_stages(::max(S, 0), S - n, u.window, u.sinks).count()) * u.n_kv;
  };
  // sums over the CTA of units and of their cost; also what lies before each thread
  struct Sum {
    long long units, cost;
  };
  auto scan = [&](long long units, long long cost, Sum& before) -> Sum {
    long long v0 = units, v1 = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x0 = __shfl_up_sync(0xFFFFFFFFu, v0, o), x1 = __shfl_up_sync(0xFFFFFFFFu, v1, o);
      if (lane >= o) v0 += x0, v1 += x1;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp][0] = v0, s_scan[warp][1] = v1;
    __syncthreads();
    Sum sum = {0, 0};
    before = {v0 - units, v1 - cost};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before.units += s_scan[w][0], before.cost += s_scan[w][1];
      sum.units += s_scan[w][0];
      sum.cost += s_scan[w][1];
    }
    return sum;
  };
  auto cost = [&](long long units) { return units ? units + (long long)kPairCost * u.n_kv : 0; };
  Sum total = {0, 0}, before;
  long long mine = 0;
  int S = 0, n = 0, q0 = 0;
  for (int r0 = 0; r0 < u.R; r0 += kChunk) {
    mine = request(r0 + tid, S, n, q0);
    const Sum sum = scan(mine, cost(mine), before);
    total.units += sum.units;
    total.cost += sum.cost;
  }
  // no more CTAs than the cost can be shared among: the parts of a split pair are then consecutive CTAs
  const int grid = (int)::min((long long)gridDim.x, ::max(total.cost, 1ll)), cta = ::min((int)blockIdx.x, grid);
  const long long cost_end = total.cost * (cta + 1) / grid;
  if (tid < 2) s_bound[tid] = total.units;  // (what no request holds is the end)
  Sum base = {0, 0};
  for (int r0 = 0; r0 < u.R; r0 += kChunk) {
    if (u.R > kChunk) mine = request(r0 + tid, S, n, q0);  // else they are still in registers
    const Sum sum = scan(mine, cost(mine), before);
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // the units before this CTA's share and before its end
      const long long rel = (e ? cost_end : total.cost * cta / grid) - base.cost - before.cost;
      if (mine && rel >= 0 && rel < cost(mine)) {
        const long long n_st = mine / u.n_kv, head = rel / (n_st + kPairCost);
        s_bound[e] = base.units + before.units + head * n_st + ::max(0ll, rel - head * (n_st + kPairCost) - kPairCost);
      }
    }
    base.units += sum.units;
    base.cost += sum.cost;
  }
  __syncthreads();
  const long long u_begin = s_bound[0];
  const int u_end = (int)(s_bound[1] - u_begin);
  const KvPlanes pl = kv_planes(u.page, D);
  const uint32_t hb = (uint32_t)kv_head_bytes(u.page, D);
  const int page_shift = __ffs(u.page) - 1;
  // where this lane's operands of the warp's 32 keys lie in a stage (shared
  // addresses), and how far on those of the second 16 are
  const int key_w = (warp % kTeam) * 32, at0 = key_w & (u.page - 1);
  const bool apart = u.page == 16;  // the second 16 keys are another page's
  const uint32_t blk0 = smem_u32(smem) + (key_w >> page_shift) * hb;
  const uint32_t at_k = blk0 + (at0 + g) * (D / 2) + q * (NB * 4), at_ks = blk0 + pl.ks + (at0 + g) * (NB * 2);
  const uint32_t at_v = blk0 + pl.vc + (at0 / 2 + q) * D + g * (NB * 4), at_vs = blk0 + pl.vs + (at0 / 2 + q) * (NB * 4);
  const uint32_t on_k = apart ? hb : 16 * (D / 2), on_ks = apart ? hb : 16 * NB * 2;
  const uint32_t on_v = apart ? hb : 8 * D, on_vs = apart ? hb : 8 * NB * 4;
  // -8 and -8 x 16 as the values' operand, in registers that the compiler does not fill anew for every use
  uint32_t off[4];
  asm volatile("mov.u32 %0, 0x80088008;\n\tmov.u32 %1, 0x80808080;\n\tmov.u32 %2, 0x80088008;\n\tmov.u32 %3, 0x80808080;"
               : "=r"(off[0]), "=r"(off[1]), "=r"(off[2]), "=r"(off[3]));

  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {  // by a whole warp
    if (ok && !__all_sync(0xFFFFFFFFu, mbar_wait(bar, parity))) {
      ok = false;
      raise(u.status, FW_KV_TIMEOUT);
    }
  };
  uint32_t it = 0, last_fill = 0;  // stages consumed; one past the last stage this warp filled
  long long chunk = total.units;  // a chunk's units
  base.units = -u_begin;
  for (int r0 = 0; r0 < u.R && base.units < u_end; r0 += kChunk) {
    if (u.R > kChunk) {
      mine = request(r0 + tid, S, n, q0);
      chunk = scan(mine, 0, before).units;
    }
    // (a request's units and a CTA's share fit 32 bits: checked on the host; what lies before the CTA's share does not matter)
    s_pref[tid] = (int)::max(::min(base.units + before.units, 1ll << 30), -(1ll << 30));
    s_len[tid] = S;
    s_new[tid] = n;
    s_tok[tid] = q0;
    base.units += chunk;
    if (tid == 0) s_pref[kChunk] = (int)::max(::min(base.units, 1ll << 30), -(1ll << 30));
    __syncthreads();
    const int from = ::max(0, s_pref[0]), to = ::min(u_end, s_pref[kChunk]);
    if (from >= to) continue;
    int k = 0;  // the request (of the chunk) that holds unit `from`
    for (int step = kChunk / 2; step; step >>= 1)
      if (s_pref[k + step] <= from) k += step;

    // Filling a stage takes two steps, so that the block table's latency is
    // nobody's: look() finds unit y's pages, one to a lane (the pages without a
    // key that some row sees are left out), several stages before issue()
    // copies them. kf: the request at or before the next y's.
    int kf = k, f_head = 0, f_id = 0;
    bool f_copy = false;
    auto look = [&](int y) {
      f_copy = false;
      if (y >= to) return;
      while (s_pref[kf + 1] <= y) ++kf;
      const int S_r = s_len[kf], first = S_r - s_new[kf];
      const Stages v = visible_stages(::max(S_r, 0), first, u.window, u.sinks);
      const int lo_key = u.window ? ::max(0, ::max(0, first) + 1 - u.window) : 0;
      const int n_st = ::max(1, v.count()), rel = y - s_pref[kf];
      f_head = rel / n_st;
      const int key = v.block(rel - f_head * n_st) * kStageKeys + (lane << page_shift);
      f_copy = lane < (kStageKeys >> page_shift) && key < S_r && (key + u.page > lo_key || key < u.sinks);
      if (f_copy) f_id = u.block_table[(int64_t)(r0 + kf) * u.max_blocks + (key >> page_shift)];
    };
    auto issue = [&](uint32_t j) {
      const int slot = j % kStages;
      bool copy = f_copy;
      if (copy && (f_id < 0 || f_id >= u.n_pages)) {
        copy = false;
        raise(u.status, FW_KV_BAD_SLOT);
      }
      const uint32_t got = __ballot_sync(0xFFFFFFFFu, copy);
      // all readers of the slot's stages before have left it. A count, not a
      // barrier's parity: this warp need not have seen the phases before, and
      // two phases apart look alike.
      if (ok && !__all_sync(0xFFFFFFFFu, wait_count(&s_left[slot], kTeam * (j / kStages)))) {
        ok = false;
        raise(u.status, FW_KV_TIMEOUT);
      }
      if (!ok) return;
      if (lane == 0) {
        uint32_t have = 0;  // a page's bit, for each 16 keys of it
#pragma unroll
        for (int w = 0; w < kStageKeys / 16; ++w) have |= (got >> ((w * 16) >> page_shift) & 1) << w;
        s_have[slot] = have;
        mbar_arrive_expect_tx(&full[slot], (uint32_t)__popc(got) * hb);
      }
      __syncwarp();
      if (copy)
        bulk_g2s(smem + slot * C::StageBytes + lane * hb, (const uint8_t*)u.cache + ((int64_t)f_id * u.n_kv + f_head) * hb, hb,
                 &full[slot]);
      last_fill = j + 1;
    };
    // the warps take turns at filling, kStages - 1 stages ahead
    const uint32_t it0 = it - from;  // the ring's count at this CTA's first unit
    if (warp < kStages - 1 && from + warp < to) {
      look(from + warp);
      issue(it + warp);
    }
    // the unit this warp fills next: at the end of the stage kStages - 1 before, one of its team's
    const int turn = 2 * (warp % kTeam) + warp / kTeam;
    int next = from + kStages - 1 + ((turn - (int)it) & (kWarps - 1));
    look(next);

    for (int x = from; x < to; ++k) {
      const int p0 = s_pref[k], p1 = s_pref[k + 1];
      if (p1 <= x) continue;
      const int S_r = s_len[k], n_r = s_new[k], first = S_r - n_r, rows = n_r * G, tok0 = s_tok[k];
      const Stages v = visible_stages(::max(S_r, 0), first, u.window, u.sinks);
      const int n_st = ::max(1, v.count());
      const int lo_key = u.window ? ::max(0, ::max(0, first) + 1 - u.window) : 0;  // the first key of the first row's window
      const int lo_edge = u.window ? lo_key + n_r : 0;  // keys below are not seen by every row
      const int stop = ::min(p1, to);
      while (x < stop) {  // one segment: the rest of this head's stages, or of this CTA's share
        const int head = (x - p0) / n_st, st0 = x - p0 - head * n_st;
        const int n_here = ::min(n_st - st0, stop - x);
        // Query rows as the 8-column operand: thread (g, q) holds row g's dims
        // 32 b + 8 q .. + 7, those of the upper nibbles a sixteenth. One tile of
        // rows stays in registers, two in shared memory.
        auto tile_q = [&](int t, uint4 (&qf)[NB]) {  // by a whole warp
          const int row = 8 * t + g;
          uint32_t most = 0;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (row < rows)
              w = *reinterpret_cast<const uint4*>((const __nv_bfloat16*)u.q + (int64_t)(tok0 + row / G) * u.q_stride +
                                                  (head * G + row % G) * D + 32 * b + 8 * q);
            float z = 0.f, lo, hi;
            for (uint32_t x : {w.x, w.y, w.z, w.w}) {
              bf16x2_to_f32(x, lo, hi);
              z += lo + hi;
            }
            z += __shfl_xor_sync(0xFFFFFFFFu, z, 1);
            z += __shfl_xor_sync(0xFFFFFFFFu, z, 2);
            if (q == 0) s_qz[row][b] = z * (-8.f / kOScale);
            most = __vmaxu2(most, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
            qf[b] = make_uint4(mul_bf16x2(w.x, kQUp), mul_bf16x2(w.y, kQUp16), mul_bf16x2(w.z, kQUp), mul_bf16x2(w.w, kQUp16));
          }
          // Products in units of 2^-69 of a row without an element of kLeast fall
          // out of fp32: made NaN, it is taken plainly at the join.
          most = __vmaxu2(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
          most = __vmaxu2(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
          most = ::max(most & 0xFFFFu, most >> 16);
          if (q == 0 && most && most < kLeast) s_qz[row][0] = __uint_as_float(0x7FC00000u);
        };
        uint4 qf[NT == 1 ? NB : 1];
        if constexpr (NT == 1) {
          tile_q(0, qf);  // every warp for itself; what they write is the same
        } else if (warp < NT) {
          uint4 w[NB];
          tile_q(warp, w);
#pragma unroll
          for (int b = 0; b < NB; ++b) *reinterpret_cast<uint4*>(s_q + ((warp * NB + b) * 32 + lane) * 16) = w[b];
        }
        __syncthreads();  // (the previous segment's buffers are no longer read either)
        // the three bf16 parts of row g's z as a 16-step operand: step k holds
        // part k / NB of block k % NB
        uint32_t qz[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          auto part = [&](int k) {
            if (k >= 3 * NB) return 0.f;
            float x = s_qz[8 * t + g][k % NB];
            for (int i = 0; i < k / NB; ++i) x -= __bfloat162float(__float2bfloat16_rn(x));
            return x;
          };
          qz[t][0] = bf16x2_bits(part(2 * q), part(2 * q + 1));
          qz[t][1] = bf16x2_bits(part(2 * q + 8), part(2 * q + 9));
        }
        auto position = [&](int row) { return row < rows ? first + row / G : -1; };  // (rows past the last see nothing)
        // mz: a row's maximum less 64 (0 before there is one); lim: what a score
        // may pass it by before it moves (-inf: there is none yet)
        float o[NT][NB][2][4] = {}, mz[NT][2], lim[NT][2], l[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) mz[t][0] = mz[t][1] = l[t][0] = l[t][1] = 0.f, lim[t][0] = lim[t][1] = -INFINITY;

        // 16 H keys of this warp, from its `half`-th 16 on. kEdge: not every row
        // sees all of them (the last keys, the window's edge) or not all are
        // there (bits of `have`); `stage`: byte offset of their stage.
        auto keys = [&](auto edge, uint32_t stage, int half, uint32_t have, int key0) {
          constexpr bool kEdge = decltype(edge)::value;
          float s[H][NT][4];
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const bool second = H == 2 ? h : half;
            const uint32_t in_k = at_k + stage + (second ? on_k : 0), in_ks = at_ks + stage + (second ? on_ks : 0);
            const Words<NB> k0 = lds<NB, 0>(in_k), k1 = lds<NB, 8 * (D / 2)>(in_k);
            const Words<NB / 2> d0 = lds<NB / 2, 0>(in_ks), d1 = lds<NB / 2, 8 * NB * 2>(in_ks);
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t z0 = NB == 4 && (q & 1) ? d0.w[NB / 2 - 1] : d0.w[0], z1 = NB == 4 && (q & 1) ? d1.w[NB / 2 - 1] : d1.w[0];
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816(s[h][t], z0, z1, z0, z1, qz[t][0], qz[t][1], zero);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const float e0 = __uint_as_float(b & 1 ? d0.w[b / 2] & 0xFFFF0000u : d0.w[b / 2] << 16);
              const float e1 = __uint_as_float(b & 1 ? d1.w[b / 2] & 0xFFFF0000u : d1.w[b / 2] << 16);
              const uint32_t x0 = k0.w[b], x1 = k1.w[b], y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                uint4 w;
                if constexpr (NT == 1)
                  w = qf[b];
                else
                  w = *reinterpret_cast<const uint4*>(s_q + ((t * NB + b) * 32 + lane) * 16);
                float c[4];
                mma16816(c, x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x00F000F0u, w.x, w.y, zero);
                mma16816(c, y0 & 0x000F000Fu, y1 & 0x000F000Fu, y0 & 0x00F000F0u, y1 & 0x00F000F0u, w.z, w.w, c);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[h][t][e] = fmaf(c[e], e < 2 ? e0 : e1, s[h][t][e]);
              }
            }
          }
          // in units of log2 and less the row's maximum as last taken
          bool moves = false;
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float& x = s[h][t][e];
                x = fmaf(x, a.scale_log2, -mz[t][e & 1]);
                if (kEdge && !((have >> h & 1) &&
                               sees(position(8 * t + 2 * q + (e & 1)), key0 + 16 * h + g + 8 * (e >> 1), u.window, u.sinks)))
                  x = -INFINITY;
                moves |= x > lim[t][e & 1];
              }
          if (__any_sync(0xFFFFFFFFu, moves)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float up = fmaxf(s[0][t][j], s[0][t][j + 2]);
                if constexpr (H == 2) up = fmaxf(up, fmaxf(s[H - 1][t][j], s[H - 1][t][j + 2]));
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) up = fmaxf(up, __shfl_xor_sync(0xFFFFFFFFu, up, d));
                // a first maximum is taken as it is, a later one only moves up
                up -= kShift;
                if (lim[t][j] != -INFINITY) up = fmaxf(up, 0.f);
                const bool none = up == -INFINITY;  // (nothing seen yet: all stays as it is)
                up = none ? 0.f : up;
                const float keep = none ? 1.f : lim[t][j] == -INFINITY ? 0.f : exp2_fast(-up);
                mz[t][j] += up;
                lim[t][j] = none ? lim[t][j] : kShift + kLazy;
                l[t][j] *= keep;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                  s[h][t][j] -= up;
                  s[h][t][j + 2] -= up;
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    o[t][b][h][j] *= keep;
                    o[t][b][h][j + 2] *= keep;
                  }
              }
          }
          // probabilities: row g, keys 2 q, 2 q + 1 (+ 8), each in two bf16 parts,
          // so that only its product with the value's scale is rounded
          uint32_t pf[H][NT][2], rest[H][NT][2];
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              float(&x)[4] = s[h][t];
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = exp2_fast(x[e]);
              l[t][0] += x[0] + x[2];
              l[t][1] += x[1] + x[3];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t lo = __float_as_uint(x[2 * e]), hi = __float_as_uint(x[2 * e + 1]);
                pf[h][t][e] = transpose8x8(__byte_perm(lo, hi, 0x7632));  // the upper halves
                rest[h][t][e] = transpose8x8(bf16x2_bits(x[2 * e] - __uint_as_float(lo & 0xFFFF0000u), x[2 * e + 1] - __uint_as_float(hi & 0xFFFF0000u)));
              }
            }
          // values
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const bool second = H == 2 ? h : half;
            const uint32_t in_v = at_v + stage + (second ? on_v : 0), in_vs = at_vs + stage + (second ? on_vs : 0);
            // which of this lane's two key pairs its row g sees, as masks of packed pairs
            uint32_t keep[NT][2];
            if constexpr (kEdge) {
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int p = position(8 * t + g), j = key0 + 16 * h + 8 * e + 2 * q;
                  keep[t][e] = (sees(p, j, u.window, u.sinks) ? 0xFFFFu : 0u) | (sees(p, j + 1, u.window, u.sinks) ? 0xFFFF0000u : 0u);
                  if (!(have >> h & 1)) keep[t][e] = 0;
                }
            }
            const Words<NB> v0 = lds<NB, 0>(in_v), v1 = lds<NB, 4 * D>(in_v);
            const Words<NB> f0 = lds<NB, 0>(in_vs), f1 = lds<NB, 4 * NB * 4>(in_vs);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              uint32_t w0[NT], w1[NT];
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                w0[t] = fma_bf16x2(pf[h][t][0], f0.w[b], mul_bf16x2(rest[h][t][0], f0.w[b]));
                w1[t] = fma_bf16x2(pf[h][t][1], f1.w[b], mul_bf16x2(rest[h][t][1], f1.w[b]));
                if constexpr (kEdge) {  // a masked key adds nothing, whatever its scale is
                  w0[t] &= keep[t][0];
                  w1[t] &= keep[t][1];
                }
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {  // dims 2 e of the lane's four (x 1) in rows g, 2 e + 1 (x 16) in rows g + 8
                const uint32_t x0 = e ? v0.w[b] >> 8 : v0.w[b], x1 = e ? v1.w[b] >> 8 : v1.w[b];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                  mma16816(o[t][b][e], x0 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x000F000Fu, x1 & 0x00F000F0u, w0[t], w1[t], o[t][b][e]);
                  mma16816(o[t][b][e], off[0], off[1], off[2], off[3], w0[t], w1[t], o[t][b][e]);
                }
              }
            }
          }
        };

        // the stages of this warp's team
#pragma unroll 1
        for (int i = (it ^ (warp / kTeam)) & 1; i < n_here; i += 2) {
          const uint32_t j = it + i;
          const int slot = j % kStages;
          wait(&full[slot], (j / kStages) & 1);
          const int key0 = v.block(st0 + i) * kStageKeys + key_w;
          const uint32_t have = ok ? s_have[slot] >> (key_w / 16) & 3 : 0, stage = slot * C::StageBytes;
#pragma unroll 1
          for (int h = 0; h < 2; h += H) {
            const int key_h = key0 + 16 * h;
            const uint32_t there = have >> h & ((1u << H) - 1);
            if (!there || key_h >= S_r) continue;
            if (there == (1u << H) - 1 && key_h + 16 * H - 1 <= first && key_h >= lo_edge)
              keys(std::false_type{}, stage, h, there, key_h);
            else
              keys(std::true_type{}, stage, h, there, key_h);
          }
          __syncwarp();
          if (lane == 0) add_release(&s_left[slot]);
          // this warp's turn: the slot of the stage before, which the other team has left by now
          if (x + i + kStages - 1 == next && next < to) {
            issue(it0 + next);
            next += kWarps;
            look(next);
          }
        }
        it += n_here;

        // -------------------------------- join the eight warps, a tile of rows at a time
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[t][j] += __shfl_xor_sync(0xFFFFFFFFu, l[t][j], d);
            const float m = lim[t][j] == -INFINITY ? -INFINITY : mz[t][j];
            if (g == 0) s_ml[warp][8 * t + 2 * q + j] = make_float2(m, l[t][j] * kLScale);
          }
        __syncthreads();
        const bool whole = n_here == n_st;
        const int part = 2 * cta + (x == 0 ? 0 : 1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          // warps 4..7 hand over to warps 0..3, whose sums the rows' threads then add
#pragma unroll
          for (int half = 1; half >= 0; --half) {
            if (warp / (kWarps / 2) == half) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int row = 8 * t + 2 * q + j;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][row].x);
                const float f = lim[t][j] == -INFINITY ? 0.f : exp2_fast(mz[t][j] - top) * kOScale, f16 = f * 0.0625f;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                  float4* at = reinterpret_cast<float4*>(join + ((warp % (kWarps / 2)) * 8 + 2 * q + j) * C::Pitch + 32 * b + 4 * g);
                  float4 y = make_float4(o[t][b][0][j] * f, o[t][b][0][j + 2] * f16, o[t][b][1][j] * f, o[t][b][1][j + 2] * f16);
                  if (half == 0) {
                    const float4 z = *at;
                    y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
                  }
                  *at = y;
                }
              }
            }
            __syncthreads();
          }
          for (int e = tid; e < 8 * (D / 4); e += kThreads) {
            const int r8 = e / (D / 4), row = 8 * t + r8, d4 = e % (D / 4);
            if (row >= rows) break;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][row].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float2 ml = s_ml[w][row];
              sum += ml.y * (ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - top));
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps / 2; ++w) {
              const float4 y = *reinterpret_cast<const float4*>(join + (w * 8 + r8) * C::Pitch + 4 * d4);
              acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
            }
            // Codes at 2^-133 and probabilities at 2^64 leave a range: products p d
            // above 2^63 are infinite and below 2^-57 are lost, and so are scores of
            // queries above 2^63 and below kLeast. A row that has
            // something infinite or NaN, or nothing above 2^-24 although not all values
            // are zero, is taken plainly: about a microsecond a key, for what no
            // model's values are. (The checks: 1 % of a call.)
            const float big = fmaxf(fmaxf(fabsf(acc.x), fabsf(acc.y)), fmaxf(fabsf(acc.z), fabsf(acc.w)));
            const uint32_t mine = D == 128 ? 0xFFFFFFFFu : 0xFFFFu << (lane & 16);
            const bool finite = big < INFINITY && acc.x == acc.x && acc.y == acc.y && acc.z == acc.z && acc.w == acc.w;
            if (ok && sum != 0.f) {
              const bool lost = !__any_sync(mine, big > 5.9e-8f * sum), some = __any_sync(mine, big != 0.f);
              if (__any_sync(mine, !finite) || lost) {
                const Segment g = {(const uint8_t*)u.cache + (int64_t)head * hb, u.block_table + (int64_t)(r0 + k) * u.max_blocks,
                                   (const __nv_bfloat16*)u.q + (int64_t)(tok0 + row / G) * u.q_stride + (head * G + row % G) * D,
                                   v, st0, n_here, S_r, first + row / G};
                if (!lost || some || has_values<D>(u, g, d4, mine)) {
                  top = plainly<D>(u, g, d4, mine, acc);
                  sum = top == -INFINITY ? 0.f : 1.f;
                  top -= kShift;
                }
              }
            }
            if (whole) {
              const float inv = sum == 0.f ? 0.f : 1.f / sum;
              __nv_bfloat16* dst = (__nv_bfloat16*)u.out + (int64_t)(tok0 + row / G) * u.out_stride + (head * G + row % G) * D + 4 * d4;
              *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2_bits(acc.x * inv, acc.y * inv), bf16x2_bits(acc.z * inv, acc.w * inv));
            } else {
              *reinterpret_cast<float4*>(a.o + ((int64_t)part * C::Rows + row) * D + 4 * d4) = acc;
              if (d4 == 0) a.ml[(int64_t)part * C::Rows + row] = make_float2(top, sum);
            }
          }
          if (t + 1 < NT) __syncthreads();
        }
        if (!whole && st0 == 0 && tid == 0) {
          // the share ends n_here units into this head; the CTA that has its last one
          SplitRecord rec;
          rec.parts = (int)(((cost_end + n_st - n_here) * grid - 1) / total.cost) - cta + 1;
          rec.slot0 = part;
          rec.slot1 = 2 * cta;
          rec.step = 2;
          rec.rows = rows;
          rec.row0 = 0;
          rec.token0 = tok0;
          rec.head0 = head * G;
          a.rec[cta] = rec;
        }
        x += n_here;
      }
    }
  }
  // copies in flight after an abandoned wait land before the CTA leaves: this
  // warp's last kStages fills are the only ones that can be
  if (!ok)
    for (uint32_t j = last_fill > (uint32_t)kStages ? last_fill - kStages : 0; j < last_fill; ++j)
      mbar_wait(&full[j % kStages], (j / kStages) & 1);
}

int decode_tiles(const fw_attn_q4_args& a) { return (int64_t)a.max_q * (a.n_q / a.n_kv) <= 8 ? 1 : 2; }

// CTAs: as many as the SMs hold, but no more than there can be units.
int decode_grid(const fw_attn_q4_args& a, int sms) {
  const int64_t most = (int64_t)a.R * a.n_kv * (((int64_t)a.max_blocks * a.page + kStageKeys - 1) / kStageKeys);
  return (int)::min((int64_t)sms * 2, most < 1 ? 1 : most);
}

template <int D, int NT>
cudaError_t launch(const DecodeArgs& d, int grid, cudaStream_t s) {
  cudaError_t e = launch_dependent(attn_decode_kernel<D, NT>, dim3(grid), dim3(kThreads), Cfg<D, NT>::SmemBytes, s, d);
  if (e == cudaSuccess) e = launch_attn_join(d.u, d.rec, d.o, d.ml, grid, 8 * NT, s);
  return e;
}

}  // namespace

cudaError_t configure_decode_attn() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto* k, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  set(attn_decode_kernel<64, 1>, Cfg<64, 1>::SmemBytes);
  set(attn_decode_kernel<64, 2>, Cfg<64, 2>::SmemBytes);
  set(attn_decode_kernel<128, 1>, Cfg<128, 1>::SmemBytes);
  set(attn_decode_kernel<128, 2>, Cfg<128, 2>::SmemBytes);
  return e;
}

int64_t decode_workspace(const fw_attn_q4_args& a, int sms) {
  const int64_t grid = decode_grid(a, sms), rows = 8 * decode_tiles(a);
  return grid * sizeof(SplitRecord) + 2 * grid * rows * (a.D * 4 + 8);
}

cudaError_t launch_attn_decode(const fw_attn_q4_args& a, void* workspace, int sms, cudaStream_t s) {
  const int nt = decode_tiles(a), grid = decode_grid(a, sms);
  DecodeArgs d;
  d.u = a;
  d.rec = static_cast<SplitRecord*>(workspace);
  d.o = reinterpret_cast<float*>(d.rec + grid);
  d.ml = reinterpret_cast<float2*>(d.o + (int64_t)2 * grid * 8 * nt * a.D);
  d.scale_log2 = a.scale * kLog2e * kOScale;  // the scores' products come in units of 2^-69
  if (a.D == 64) return nt == 1 ? launch<64, 1>(d, grid, s) : launch<64, 2>(d, grid, s);
  return nt == 1 ? launch<128, 1>(d, grid, s) : launch<128, 2>(d, grid, s);
}

}  // namespace fw
