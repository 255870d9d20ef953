// The attention side of a layer around its cache: the step's plan (block
// tables, slots, positions), the norms and rotation of queries and keys with
// the store into the 4-bit cache, and the read-back.
#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "kvcache.cuh"

namespace fw {
namespace {

using namespace dev;

// ------------------------------------------------------------- the plan
// Two running sums over the requests decide everything: of the new tokens
// (which request a token belongs to) and of the fresh pages (which entry of
// the free list a block takes). Every CTA makes both sums for itself -- R
// lengths are a few KB from L2 -- so one launch without any wait between CTAs
// is enough; it then fills its own kPlanTokens tokens. The thread of the token
// that opens a fresh page also writes that page's block-table entry, so a
// request of any length is spread over the grid. What bounds it is latency:
// one launch, two dependent loads and a scan of the lengths.
constexpr int kPlanThreads = 512, kPlanItems = 4, kPlanChunk = kPlanThreads * kPlanItems;
constexpr int kPlanTokens = 1024;  // tokens per CTA
constexpr int kMaxLen = 1 << 30;
constexpr int kMaxSlot = 0x7FFFFFFF;  // past every cache: these have fewer positions

struct PlanArgs {
  const int32_t *ctx, *fresh, *free_pages, *free_used;
  int32_t* table;
  int R, max_blocks, n_free, page_shift, T_cap;
  int32_t *q_start, *seq_lens, *req, *pos, *slot, *counts;
};

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
  __shared__ int s_start[kPlanChunk + 1];  // first new token of each request of the chunk (clamped to kMaxLen)
  __shared__ int s_ctx[kPlanChunk];
  __shared__ int s_page[kPlanChunk];       // free-list index of its first fresh page
  __shared__ longlong2 s_warp[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = blockIdx.x * kPlanTokens, t1 = ::min(a.T_cap, t0 + kPlanTokens);
  const int P = 1 << a.page_shift;
  const bool first_cta = blockIdx.x == 0;
  // 64-bit sums: no lengths that pass the check below overflow them
  long long tokens = 0, pages = a.free_used ? ::max(0, *a.free_used) : 0;
  int bits = 0;
  for (int r0 = 0; r0 < a.R; r0 += kPlanChunk) {
    if (!first_cta && tokens >= t1) return;  // all of this CTA's tokens are done
    int c[kPlanItems], n_new[kPlanItems], n_pages[kPlanItems];
    long long sum_t = 0, sum_p = 0;
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) {
      const int r = r0 + tid * kPlanItems + i;
      int n = 0;
      c[i] = 0;
      if (r < a.R) {
        c[i] = a.ctx[r];
        n = a.fresh[r];
        if (c[i] < 0 || n < 0 || c[i] > kMaxLen || n > kMaxLen - c[i]) {
          bits |= FW_KV_BAD_LENGTH;
          c[i] = n = 0;
        }
        if ((c[i] + n + P - 1) >> a.page_shift > a.max_blocks) bits |= FW_KV_TABLE_FULL;
      }
      n_new[i] = n;
      n_pages[i] = ((c[i] + n + P - 1) >> a.page_shift) - ((c[i] + P - 1) >> a.page_shift);
      sum_t += n;
      sum_p += n_pages[i];
    }
    longlong2 inc = make_longlong2(sum_t, sum_p);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long ut = __shfl_up_sync(0xFFFFFFFFu, inc.x, o), up = __shfl_up_sync(0xFFFFFFFFu, inc.y, o);
      if (lane >= o) {
        inc.x += ut;
        inc.y += up;
      }
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    long long before_t = tokens + inc.x - sum_t, before_p = pages + inc.y - sum_p;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      const longlong2 u = s_warp[w];
      if (w < warp) {
        before_t += u.x;
        before_p += u.y;
      }
      tokens += u.x;
      pages += u.y;
    }
    const int n_here = ::min(kPlanChunk, a.R - r0);
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) {
      const int k = tid * kPlanItems + i;
      const int start = (int)::min(before_t, (long long)kMaxLen);
      s_start[k] = start;
      s_ctx[k] = c[i];
      s_page[k] = (int)::min(before_p, (long long)kMaxLen);
      if (first_cta && k < n_here) {
        a.q_start[r0 + k] = start;
        a.seq_lens[r0 + k] = c[i] + n_new[i];
      }
      before_t += n_new[i];
      before_p += n_pages[i];
    }
    const int end = (int)::min(tokens, (long long)kMaxLen);
    if (tid == 0) s_start[n_here] = end;
    __syncthreads();
    const int lo = ::max(t0, s_start[0]), hi = ::min(t1, end);
    for (int t = lo + tid; t < hi; t += kPlanThreads) {
      int l = 0, h = n_here;  // the last request that starts at or before t
      while (h - l > 1) {
        const int m = (l + h) >> 1;
        if (s_start[m] <= t) l = m; else h = m;
      }
      const int r = r0 + l, pos = s_ctx[l] + t - s_start[l];
      const int blk = pos >> a.page_shift, have = (s_ctx[l] + P - 1) >> a.page_shift;
      int page = -1;
      if (blk < a.max_blocks) {
        int32_t* entry = a.table + (int64_t)r * a.max_blocks + blk;
        if (blk < have) {
          page = *entry;
        } else {
          const int f = s_page[l] + blk - have;
          if (f < a.n_free) page = a.free_pages[f];
          if ((pos & (P - 1)) == 0) *entry = page;
        }
      }
      a.req[t] = r;
      a.pos[t] = pos;
      // (an id that no cache has must not come out as a slot that one has)
      a.slot[t] = page < 0 ? -1 : page > kMaxSlot >> a.page_shift ? kMaxSlot : (page << a.page_shift) + (pos & (P - 1));
    }
    __syncthreads();
  }
  const int total = (int)::min(tokens, (long long)kMaxLen);
  for (int t = ::max(t0, total) + tid; t < t1; t += kPlanThreads) a.req[t] = a.pos[t] = a.slot[t] = -1;
  if (first_cta) {
    const int used = (int)::min(pages, (long long)kMaxLen);
    if (used > a.n_free) bits |= FW_KV_POOL_EMPTY;
    if (total > a.T_cap) bits |= FW_KV_TOKENS_FULL;
    bits = __syncthreads_or(bits & FW_KV_BAD_LENGTH) ? bits | FW_KV_BAD_LENGTH : bits;
    bits = __syncthreads_or(bits & FW_KV_TABLE_FULL) ? bits | FW_KV_TABLE_FULL : bits;
    if (tid == 0) {
      a.q_start[a.R] = total;
      a.counts[0] = total;
      a.counts[1] = used;
      a.counts[2] = bits;
    }
  }
}

// ------------------------------------------------------------- norms, rotation, store
// A head's row of D values lies in D / 8 lanes, 16 bytes each, so its sum of
// squares, its rotation partners and a 4-bit block's extreme are a few
// shuffles away. A warp takes kRows rows per lane group of ONE token (its
// queries, then keys, then values, as one row index), so every row's load is
// in flight before the first sum, and the cosines and sines are loaded once
// for all of them and already multiplied by the norm's weights:
//   y = (x (w cos) + x' (w' sin)) / rms(x)
// At few tokens the chain of loads (position -> table row) is what it takes:
// 4.4 us for one token with the store and its read-back (1 row a group 3.8, 4
// rows 6.1). At many, instructions: 4096 tokens of 32 + 4 + 4 rows of 128
// take 28 us, of which moving them alone is 11, the table's rows and weights 7,
// the rows' arithmetic 10 (1 row a group 40, 4 rows 30; a persistent grid with
// the next token's rows loaded ahead 41: too few warps to hide the arithmetic).
constexpr int kRopeWarps = 8, kRopeRows = 2;  // warps of a CTA at most

struct RopeArgs {
  fw_qk_norm_rope_args u;
  int rows;        // n_q + n_kv, + n_kv when storing
  int page_shift;
  uint32_t head_bytes;
};

// One row's 4-bit block halves: the scale of the 4 lanes' 32 values (already
// bf16) and this lane's 8 codes, x / d rounded half to even. The scale is the
// element of largest magnitude (the positive one of a tie) over -8: exact in
// bf16 for bf16 values (from 2^-123 on). No quotient is needed to know how x / d rounds: with
// X, Y of 8 bits, x / d and a half-integer h / 2 from 1/2 on differ by
// |2 X 2^a - h Y| / 2 Y with a >= -2, so by nothing or by 2^-10 or more. x times
// 1 / d, rounded to a multiple of 2^-11, is on the right side of it or on it.
constexpr float kSnap = 6144.f;      // 1.5 x 2^12: sums with it are multiples of 2^-11
constexpr float kWhole = 12582912.f;  // 1.5 x 2^23: of 1, and the low bits of the sum are the whole number

__device__ __forceinline__ float quantise8(const float (&x)[8], uint32_t (&code)[8]) {
  float hi = x[0], lo = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    hi = max_nan(hi, x[i]);
    lo = min_nan(lo, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    hi = max_nan(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    lo = min_nan(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
  }
  const float d = (hi >= -lo ? hi : lo) * -0.125f;
  if (fabsf(d) > 1e-30f && fabsf(d) < 1e30f) {
    const float r = __fdiv_rn(1.f, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // |x| <= 8 |d|: only an extreme of the other sign passes what a code holds
      const float t = fminf(__fadd_rn(__fadd_rn(__fmul_rn(x[i], r), kSnap), -kSnap), 7.f);
      code[i] = __float_as_uint(__fadd_rn(t, kWhole + 8.f)) & 15;
    }
  } else {  // zeros, what is not finite, and where 1 / d would not do
#pragma unroll
    for (int i = 0; i < 8; ++i)
      code[i] = d != 0.f ? (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(x[i], d)) + 8.f, 0.f), 15.f) : 8;
  }
  return d;
}

template <int D>
__global__ void __launch_bounds__(kRopeWarps * 32, 5) qk_norm_rope_kernel(RopeArgs a) {
  constexpr int L = D / 8, Groups = 32 / L, NB = D / kKvBlock;  // lanes of a row, rows side by side in a warp
  const fw_qk_norm_rope_args& u = a.u;
  const int lane = threadIdx.x & 31, grp = lane / L, l = lane % L, half = u.rot / 2;
  const int64_t t = blockIdx.x;
  const int base = (int)(blockIdx.y * (blockDim.x / 32) + threadIdx.x / 32) * (Groups * kRopeRows), row0 = base + grp;
  pdl_wait();
  pdl_launch_dependents();
  if (base >= a.rows) return;  // a whole warp
  const bool first = l == 0 && row0 == 0, turns = 8 * l < u.rot, low = 8 * l < half;
  const bool queries = base + Groups * kRopeRows <= u.n_q;  // all of the warp's rows are

  uint4 raw[kRopeRows];
#pragma unroll
  for (int i = 0; i < kRopeRows; ++i) {
    const int r = row0 + i * Groups;
    const __nv_bfloat16* src = (const __nv_bfloat16*)u.q + t * u.q_stride + r * D;
    if (!queries && r >= u.n_q)
      src = r < u.n_q + u.n_kv ? (const __nv_bfloat16*)u.k + t * u.k_stride + (r - u.n_q) * D
                               : (const __nv_bfloat16*)u.v + t * u.v_stride + (r - u.n_q - u.n_kv) * D;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (r < a.rows) raw[i] = *reinterpret_cast<const uint4*>(src + 8 * l);
  }
  int slot = -1, pos = 0;
  if (u.cache && (!queries || first)) slot = u.slots[t];
  if (turns) {
    pos = u.positions[t];
    if (pos < 0 || pos >= u.n_pos) {
      // a padding row (-1) keeps position 0's rotation: nothing reads it
      if (pos != -1 && first) raise(u.status, FW_KV_BAD_POSITION);
      pos = 0;
    }
  }
  // The lane whose dims are this one's partners (shfl reads it mod 32), and
  // those dims: with interleaved pairs the lane has them itself.
  const int other = u.interleaved || !turns ? l : low ? l + half / 8 : l - half / 8;
  // What a row's values are multiplied by: the norm's weight and the cosine,
  // and for its partners' the weight there and the signed sine. The same for
  // all of the token's queries, and for all of its keys.
  float cw[8], sw[8];
  const float* made_for = nullptr;
  bool made = false;
  auto factors = [&](const float* w) {
    if (made && made_for == w) return;
    made = true;
    made_for = w;
#pragma unroll
    for (int j = 0; j < 8; ++j) cw[j] = 1.f, sw[j] = 0.f;
    if (turns) {
      const float* row = u.cos_sin + (int64_t)pos * u.rot;
      if (u.interleaved) {
        const float4 c = *reinterpret_cast<const float4*>(row + 4 * l), s = *reinterpret_cast<const float4*>(row + half + 4 * l);
        cw[0] = cw[1] = c.x; cw[2] = cw[3] = c.y; cw[4] = cw[5] = c.z; cw[6] = cw[7] = c.w;
        sw[1] = s.x; sw[3] = s.y; sw[5] = s.z; sw[7] = s.w;
        sw[0] = -s.x; sw[2] = -s.y; sw[4] = -s.z; sw[6] = -s.w;
      } else {
        const float* at = row + (low ? 8 * l : 8 * l - half);
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const float4 c = *reinterpret_cast<const float4*>(at + j), s = *reinterpret_cast<const float4*>(at + half + j);
          cw[j] = c.x; cw[j + 1] = c.y; cw[j + 2] = c.z; cw[j + 3] = c.w;
          sw[j] = low ? -s.x : s.x; sw[j + 1] = low ? -s.y : s.y; sw[j + 2] = low ? -s.z : s.z; sw[j + 3] = low ? -s.w : s.w;
        }
      }
    }
    if (w) {
      const float4 w0 = *reinterpret_cast<const float4*>(w + 8 * l), w1 = *reinterpret_cast<const float4*>(w + 8 * l + 4);
      const float4 p0 = *reinterpret_cast<const float4*>(w + 8 * other), p1 = *reinterpret_cast<const float4*>(w + 8 * other + 4);
      cw[0] *= w0.x; cw[1] *= w0.y; cw[2] *= w0.z; cw[3] *= w0.w;
      cw[4] *= w1.x; cw[5] *= w1.y; cw[6] *= w1.z; cw[7] *= w1.w;
      if (u.interleaved) {
        sw[0] *= p0.y; sw[1] *= p0.x; sw[2] *= p0.w; sw[3] *= p0.z;
        sw[4] *= p1.y; sw[5] *= p1.x; sw[6] *= p1.w; sw[7] *= p1.z;
      } else {
        sw[0] *= p0.x; sw[1] *= p0.y; sw[2] *= p0.z; sw[3] *= p0.w;
        sw[4] *= p1.x; sw[5] *= p1.y; sw[6] *= p1.z; sw[7] *= p1.w;
      }
    }
  };
  auto unpack = [](uint4 v, float (&x)[8]) {
    bf16x2_to_f32(v.x, x[0], x[1]);
    bf16x2_to_f32(v.y, x[2], x[3]);
    bf16x2_to_f32(v.z, x[4], x[5]);
    bf16x2_to_f32(v.w, x[6], x[7]);
  };
  auto swap_halves = [](uint32_t v) { return __funnelshift_l(v, v, 16); };
  // one row of queries or keys, normed and rotated, in bf16
  auto turn = [&](uint4 in, bool norm) {
    uint4 far;
    if (u.interleaved) {
      far = make_uint4(swap_halves(in.x), swap_halves(in.y), swap_halves(in.z), swap_halves(in.w));
    } else {
      const int from = (lane & ~(L - 1)) + other;
      far.x = __shfl_sync(0xFFFFFFFFu, in.x, from);
      far.y = __shfl_sync(0xFFFFFFFFu, in.y, from);
      far.z = __shfl_sync(0xFFFFFFFFu, in.z, from);
      far.w = __shfl_sync(0xFFFFFFFFu, in.w, from);
    }
    float x[8], y[8], sum = 0.f, inv = 1.f;
    unpack(in, x);
    unpack(far, y);
    if (u.q_norm || u.k_norm) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += x[j] * x[j];
#pragma unroll
      for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      if (norm) inv = rsqrtf(sum * (1.f / D) + u.eps);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] *= cw[j];
      if (turns) x[j] = fmaf(y[j], sw[j], x[j]);
      x[j] *= inv;
    }
    return make_uint4(bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]), bf16x2_bits(x[4], x[5]), bf16x2_bits(x[6], x[7]));
  };
  __nv_bfloat16* const q_out = (__nv_bfloat16*)u.q_out + t * u.q_out_stride + 8 * l;
  // the slot is this token's place in a page; the warp of the first row says if there is none
  uint8_t* block = nullptr;  // the token's page block of head 0
  if (slot >= 0 && slot >> a.page_shift < u.n_pages)
    block = (uint8_t*)u.cache + (int64_t)(slot >> a.page_shift) * u.n_kv * a.head_bytes;
  else if (slot != -1 && first)
    raise(u.status, FW_KV_BAD_SLOT);
  if (queries) {
    factors(u.q_norm);
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i)
      *reinterpret_cast<uint4*>(q_out + (row0 + i * Groups) * D) = turn(raw[i], u.q_norm != nullptr);
    return;
  }
  const int at = slot & (u.page - 1);
  const KvPlanes p = kv_planes(u.page, D);
#pragma unroll
  for (int i = 0; i < kRopeRows; ++i) {
    const int r = row0 + i * Groups;
    const bool is_q = r < u.n_q, is_v = r >= u.n_q + u.n_kv;
    const float* w = is_q ? u.q_norm : u.k_norm;
    if (!is_v) factors(w);
    uint4 o4 = turn(raw[i], w != nullptr);
    if (is_v) o4 = raw[i];
    if (is_q)
      *reinterpret_cast<uint4*>(q_out + r * D) = o4;
    else if (!is_v && u.k_out)
      *reinterpret_cast<uint4*>((__nv_bfloat16*)u.k_out + t * u.k_out_stride + (r - u.n_q) * D + 8 * l) = o4;
    if (!u.cache) continue;
    float x[8];
    unpack(o4, x);
    uint32_t c[8];
    const float d = quantise8(x, c);
    if (is_q || r >= a.rows || !block) continue;
    uint8_t* to = block + (is_v ? r - u.n_q - u.n_kv : r - u.n_q) * a.head_bytes;
    const int b = l / 4, q = l % 4;
    const __nv_bfloat16 db = __float2bfloat16_rn(d);
    if (!is_v) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) word |= c[j] << (4 * (j / 2) + 16 * (j % 2));
      reinterpret_cast<uint32_t*>(to + at * (D / 2))[q * NB + b] = word;
      if (q == 0) reinterpret_cast<__nv_bfloat16*>(to + p.ks)[at * NB + b] = db;
    } else {
      uint16_t* codes = reinterpret_cast<uint16_t*>(to + p.vc + (at / 2) * D);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        codes[2 * ((2 * q + k) * NB + b) + (at & 1)] = (uint16_t)(c[4 * k] | c[4 * k + 1] << 4 | c[4 * k + 2] << 8 | c[4 * k + 3] << 12);
      if (q == 0) reinterpret_cast<__nv_bfloat16*>(to + p.vs)[2 * ((at / 2) * NB + b) + (at & 1)] = db;
    }
  }
}

// ------------------------------------------------------------- read-back
// D / 8 lanes per (token, head), one 8-dim word of K and two half words of V
// each. Bound by the bf16 values it writes.
template <int D>
__global__ void __launch_bounds__(256)
    kv_export_kernel(const uint8_t* cache, int n_pages, int n_kv, int page, const int32_t* slots, int64_t rows,
                     __nv_bfloat16* k, __nv_bfloat16* v, int32_t* status) {
  constexpr int L = D / 8, NB = D / kKvBlock;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, row = i / L;
  const int l = (int)(i % L), b = l / 4, q = l % 4;
  if (row >= rows) return;
  const int head = (int)(row % n_kv), slot = slots[row / n_kv];
  uint4 ko = make_uint4(0, 0, 0, 0), vo = ko;
  if (slot >= 0 && slot / page < n_pages) {
    const uint8_t* base = cache + ((int64_t)(slot / page) * n_kv + head) * kv_head_bytes(page, D);
    const KvPlanes p = kv_planes(page, D);
    const int at = slot % page;
    const uint32_t kw = reinterpret_cast<const uint32_t*>(base + at * (D / 2))[q * NB + b];
    const float kd = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base + p.ks)[at * NB + b]);
    const uint16_t* vc = reinterpret_cast<const uint16_t*>(base + p.vc + (at / 2) * D);
    const uint32_t vw = vc[2 * ((2 * q) * NB + b) + (at & 1)] | (uint32_t)vc[2 * ((2 * q + 1) * NB + b) + (at & 1)] << 16;
    const float vd = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base + p.vs)[2 * ((at / 2) * NB + b) + (at & 1)]);
    auto pair = [](uint32_t w, int n0, int n1, float d) {
      return bf16x2_bits((float)((int)(w >> (4 * n0) & 15) - 8) * d, (float)((int)(w >> (4 * n1) & 15) - 8) * d);
    };
    ko = make_uint4(pair(kw, 0, 4, kd), pair(kw, 1, 5, kd), pair(kw, 2, 6, kd), pair(kw, 3, 7, kd));
    vo = make_uint4(pair(vw, 0, 1, vd), pair(vw, 2, 3, vd), pair(vw, 4, 5, vd), pair(vw, 6, 7, vd));
  } else if (slot != -1 && l == 0 && head == 0) {
    raise(status, FW_KV_BAD_SLOT);
  }
  *reinterpret_cast<uint4*>(k + row * D + 8 * l) = ko;
  *reinterpret_cast<uint4*>(v + row * D + 8 * l) = vo;
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

const char* kv_format_error(int n_kv, int page, int64_t n_pages) {
  if (n_kv < 1 || n_kv > 1024) return "4-bit cache: need 1 <= n_kv <= 1024";
  if (page != 16 && page != 32 && page != 64 && page != 128) return "4-bit cache: page must be 16, 32, 64 or 128 positions";
  if (n_pages < 1 || n_pages * page > 0x7FFFFFFFll) return "4-bit cache: need 1 <= n_pages and n_pages * page < 2^31";
  return nullptr;
}

// Refuses devices other than sm_103 (the only code in this library), once per device.
fw_status check_device(const char* text) {
  static std::atomic<bool> ok[64] = {};
  int dev = 0, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess && ok[dev]) return FW_OK;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e != cudaSuccess) return set_cuda_error(e, text);
  if (major != 10 || minor != 3) return set_error(FW_EUNSUPPORTED, text);
  ok[dev] = true;
  return FW_OK;
}

}  // namespace fw

using namespace fw;

extern "C" fw_status fw_kv_plan(const int32_t* cached_lens, const int32_t* new_lens, int32_t R, int32_t page,
                                int32_t* block_table, int32_t max_blocks, const int32_t* free_pages, int32_t n_free,
                                const int32_t* free_used, int32_t T_cap, int32_t* q_start, int32_t* seq_lens,
                                int32_t* requests, int32_t* positions, int32_t* slots, int32_t* counts, void* stream) {
  if (R < 0 || R > (1 << 20)) return set_error(FW_EINVAL, "fw_kv_plan: need 0 <= R <= 2^20");
  if (page != 16 && page != 32 && page != 64 && page != 128)
    return set_error(FW_EINVAL, "fw_kv_plan: page must be 16, 32, 64 or 128 positions");
  if (max_blocks < 1 || n_free < 0 || T_cap < 1 || T_cap > (1 << 30))
    return set_error(FW_EINVAL, "fw_kv_plan: need max_blocks >= 1, n_free >= 0 and 1 <= T_cap <= 2^30");
  if (!q_start || !counts || !requests || !positions || !slots ||
      (R > 0 && (!cached_lens || !new_lens || !block_table || !seq_lens)) || (n_free > 0 && !free_pages))
    return set_error(FW_EINVAL, "fw_kv_plan: null pointer");
  for (const void* p : {(const void*)cached_lens, (const void*)new_lens, (const void*)block_table, (const void*)free_pages,
                        (const void*)free_used, (const void*)q_start, (const void*)seq_lens, (const void*)requests,
                        (const void*)positions, (const void*)slots, (const void*)counts})
    if (!aligned(p, 4)) return set_error(FW_EINVAL, "fw_kv_plan: pointers need 4-byte alignment");
  if (free_used && free_used >= counts && free_used < counts + 3)
    return set_error(FW_EINVAL, "fw_kv_plan: free_used must not lie in this call's counts (use two buffers in turn)");
  if (fw_status st = check_device("fw_kv_plan: needs an sm_103 device"); st != FW_OK) return st;
  PlanArgs a = {cached_lens, new_lens, free_pages, free_used, block_table, R, max_blocks, n_free, 0, T_cap,
                q_start, seq_lens, requests, positions, slots, counts};
  while ((1 << a.page_shift) < page) ++a.page_shift;
  const cudaError_t e = dev::launch_dependent(plan_kernel, dim3((T_cap + kPlanTokens - 1) / kPlanTokens), dim3(kPlanThreads), 0,
                                              static_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return set_cuda_error(e, "fw_kv_plan: launch");
  return FW_OK;
}

extern "C" fw_status fw_qk_norm_rope(const fw_qk_norm_rope_args* u, void* stream) {
  if (!u) return set_error(FW_EINVAL, "fw_qk_norm_rope: null argument struct");
  if (u->D != 64 && u->D != 128) return set_error(FW_EUNSUPPORTED, "fw_qk_norm_rope: D must be 64 or 128");
  if (u->T < 0 || u->n_q < 1 || u->n_q > 1024 || u->n_kv < 1 || u->n_kv > 1024)
    return set_error(FW_EINVAL, "fw_qk_norm_rope: need T >= 0 and 1 <= n_q, n_kv <= 1024");
  if (u->rot < 0 || u->rot > u->D || u->rot % 16 || (u->interleaved != 0 && u->interleaved != 1))
    return set_error(FW_EINVAL, "fw_qk_norm_rope: rot must be a multiple of 16 in [0, D], interleaved 0 or 1");
  if (!(u->eps >= 0.f)) return set_error(FW_EINVAL, "fw_qk_norm_rope: eps must not be negative");
  if (u->cache) {
    if (const char* e = kv_format_error(u->n_kv, u->page, u->n_pages)) return set_error(FW_EINVAL, e);
  }
  if (u->T == 0) return FW_OK;
  if (!u->q || !u->k || !u->q_out || (!u->k_out && !u->cache) || (u->cache && (!u->v || !u->slots)))
    return set_error(FW_EINVAL, "fw_qk_norm_rope: null pointer (k_out may be null only when a cache is given, which needs v and slots)");
  if (u->rot && (!u->positions || !u->cos_sin || u->n_pos < 1))
    return set_error(FW_EINVAL, "fw_qk_norm_rope: a rotation needs positions and a cos_sin table");
  const int64_t qw = (int64_t)u->n_q * u->D, kw = (int64_t)u->n_kv * u->D;
  if (u->q_stride < qw || u->k_stride < kw || u->q_out_stride < qw || (u->k_out && u->k_out_stride < kw) ||
      (u->cache && u->v_stride < kw) || u->q_stride % 8 || u->k_stride % 8 || u->q_out_stride % 8 ||
      (u->k_out && u->k_out_stride % 8) || (u->cache && u->v_stride % 8))
    return set_error(FW_EINVAL, "fw_qk_norm_rope: token strides must cover the heads and be multiples of 8 elements");
  for (const void* p : {u->q, u->k, u->v, (const void*)u->q_norm, (const void*)u->k_norm, (const void*)u->cos_sin,
                        (const void*)u->q_out, (const void*)u->k_out, (const void*)u->cache})
    if (!aligned(p, 16)) return set_error(FW_EINVAL, "fw_qk_norm_rope: tensors need 16-byte alignment");
  if (!aligned(u->positions, 4) || !aligned(u->slots, 4) || !aligned(u->status, 4))
    return set_error(FW_EINVAL, "fw_qk_norm_rope: positions, slots and status need 4-byte alignment");
  if (fw_status st = check_device("fw_qk_norm_rope: needs an sm_103 device"); st != FW_OK) return st;
  RopeArgs a;
  a.u = *u;
  a.rows = u->n_q + u->n_kv + (u->cache ? u->n_kv : 0);
  a.head_bytes = u->cache ? (uint32_t)kv_head_bytes(u->page, u->D) : 0;
  a.page_shift = 0;
  while (u->cache && (1 << a.page_shift) < u->page) ++a.page_shift;
  // a token's rows on the warps of one CTA, or of as few as hold them, evenly
  const int per_warp = 32 / (u->D / 8) * kRopeRows, tasks = (a.rows + per_warp - 1) / per_warp;
  const int ctas = (tasks + kRopeWarps - 1) / kRopeWarps, warps = (tasks + ctas - 1) / ctas;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dev::launch_dependent(u->D == 64 ? qk_norm_rope_kernel<64> : qk_norm_rope_kernel<128>,
                                              dim3(u->T, ctas), dim3(warps * 32), 0, s, a);
  if (e != cudaSuccess) return set_cuda_error(e, "fw_qk_norm_rope: launch");
  return FW_OK;
}

extern "C" fw_status fw_kv_export(const void* cache, int32_t n_pages, int32_t n_kv, int32_t D, int32_t page,
                                  const int32_t* slots, int32_t T, void* k, void* v, int32_t* status, void* stream) {
  if (D != 64 && D != 128) return set_error(FW_EUNSUPPORTED, "fw_kv_export: D must be 64 or 128");
  if (const char* e = kv_format_error(n_kv, page, n_pages)) return set_error(FW_EINVAL, e);
  if (T < 0) return set_error(FW_EINVAL, "fw_kv_export: T must not be negative");
  if (T == 0) return FW_OK;
  if (!cache || !slots || !k || !v) return set_error(FW_EINVAL, "fw_kv_export: null pointer");
  if (!aligned(cache, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !aligned(status, 4))
    return set_error(FW_EINVAL, "fw_kv_export: cache, k and v need 16-byte, slots and status 4-byte alignment");
  if (fw_status st = check_device("fw_kv_export: needs an sm_103 device"); st != FW_OK) return st;
  const int64_t rows = (int64_t)T * n_kv, ctas = (rows * (D / 8) + 255) / 256;
  if (ctas > 0x7FFFFFFF) return set_error(FW_EINVAL, "fw_kv_export: too many rows for one launch");
  const cudaError_t e = dev::launch_dependent(D == 64 ? kv_export_kernel<64> : kv_export_kernel<128>, dim3((unsigned)ctas),
                                              dim3(256), 0, static_cast<cudaStream_t>(stream), (const uint8_t*)cache,
                                              n_pages, n_kv, page, slots, rows, (__nv_bfloat16*)k, (__nv_bfloat16*)v, status);
  if (e != cudaSuccess) return set_cuda_error(e, "fw_kv_export: launch");
  return FW_OK;
}
