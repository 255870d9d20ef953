// Joins the partial results of rows whose keys several CTAs shared:
//   o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i
// A row's D / 4 lanes read 16 bytes each. With few rows (decode) the lane groups
// of a CTA share a row's parts; with many (prefill) every group has a row of
// its own. Bound by launch and latency: 2-4 us of a call (48 drafts of 16 rows
// 26.2 us; with a CTA a row, four waves of them, 29.7).
#include "attn.cuh"

namespace fw {
namespace {

using namespace dev;

constexpr int kThreads = 256;
// Where groups share rows: rows of a CTA. Four of 16 rows if there are pairs
// enough that a record has few parts, or prompts in the call (few records then
// have any): the records' CTAs are one wave (48 drafts 26.2 us a call, a row a CTA
// 29.7; windowed prompts 53.5, 57.4). Else one, so that many parts are read at
// once (one token of 16 rows over 68,000 keys: 304 parts, 38 us instead of 93).
constexpr int kFewParts = 4;  // on average

struct JoinArgs {
  const SplitRecord* rec;
  const float* o;
  const float2* ml;
  __nv_bfloat16* out;
  int64_t out_stride;
  int rows_max, G;
  int here;  // kShare: rows of a CTA
};

template <int D, bool kShare>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(JoinArgs a) {
  constexpr int L = D / 4, Groups = kThreads / L;
  __shared__ float4 s_o[kShare ? kThreads : 1];
  __shared__ float2 s_ml[Groups];
  pdl_wait();
  pdl_launch_dependents();
  const SplitRecord rec = a.rec[blockIdx.x];
  const int l = threadIdx.x % L, grp = threadIdx.x / L;
  const int here = kShare ? a.here : Groups, share = Groups / here;  // rows of this CTA, groups of a row
  const int row = blockIdx.y * here + grp / share, first = grp % share;
  if (rec.parts == 0 || (!kShare && row >= rec.rows)) return;
  float m = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = row < rec.rows ? first : rec.parts; i < rec.parts; i += kShare ? share : 1) {
    const int64_t at = (int64_t)(i == 0 ? rec.slot0 : rec.slot1 + i * rec.step) * a.rows_max + row;
    const float2 ml = __ldcg(a.ml + at);
    // a part in which the row saw nothing has no output; NaN has to go on
    if (ml.x == -INFINITY && ml.y == 0.f) continue;
    const float4 o = __ldcg(reinterpret_cast<const float4*>(a.o + at * D) + l);
    const float top = fmaxf(m, ml.x), keep = m == -INFINITY ? 0.f : exp2_fast(m - top);
    const float f = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - top);
    m = top;
    sum = sum * keep + ml.y * f;
    acc.x = acc.x * keep + o.x * f;
    acc.y = acc.y * keep + o.y * f;
    acc.z = acc.z * keep + o.z * f;
    acc.w = acc.w * keep + o.w * f;
  }
  if constexpr (kShare) {
    s_o[threadIdx.x] = acc;
    if (l == 0) s_ml[grp] = make_float2(m, sum);
    __syncthreads();
    if (first || row >= rec.rows) return;
    float top = -INFINITY;
    for (int i = 0; i < share; ++i) top = fmaxf(top, s_ml[grp + i].x);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    sum = 0.f;
    for (int i = 0; i < share; ++i) {
      const float2 ml = s_ml[grp + i];
      const float f = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - top);
      const float4 o = s_o[(grp + i) * L + l];
      sum += ml.y * f;
      acc.x += o.x * f;
      acc.y += o.y * f;
      acc.z += o.z * f;
      acc.w += o.w * f;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int n = rec.row0 + row;
  __nv_bfloat16* dst = a.out + (int64_t)(rec.token0 + n / a.G) * a.out_stride + (rec.head0 + n % a.G) * D + 4 * l;
  *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2_bits(acc.x * inv, acc.y * inv), bf16x2_bits(acc.z * inv, acc.w * inv));
}

}  // namespace

cudaError_t launch_attn_join(const fw_attn_q4_args& a, const SplitRecord* rec, const float* o, const float2* ml, int records,
                             int rows_max, cudaStream_t s) {
  const bool share = rows_max <= kDecodeRows;
  const bool prompts = (int64_t)a.max_q * (a.n_q / a.n_kv) > kDecodeRows;
  const int here = rows_max > 8 && (prompts || (int64_t)a.R * a.n_kv * kFewParts >= records) ? 4 : 1;
  const JoinArgs j = {rec, o, ml, (__nv_bfloat16*)a.out, a.out_stride, rows_max, a.n_q / a.n_kv, here};
  const int groups = kThreads / (a.D / 4);
  const dim3 grid(records, rows_max / (share ? here : groups));
  if (a.D == 64) return launch_dependent(share ? attn_join_kernel<64, true> : attn_join_kernel<64, false>, grid, dim3(kThreads), 0, s, j);
  return launch_dependent(share ? attn_join_kernel<128, true> : attn_join_kernel<128, false>, grid, dim3(kThreads), 0, s, j);
}

}  // namespace fw
