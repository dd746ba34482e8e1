// Attention of one new token a sequence over the paged key-value cache.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp2(t_j - max t),  t_j = (scale log2 e) q.k_j
//
// One CTA a (sequence, query head); its warps take the tokens in turn, each with its own running
// maximum, sum and fp32 accumulator, joined through shared memory at the end.
#include "decoder.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float cache_value(const CacheDev& c, const uint8_t* p, int64_t row, int d, float unit) {
  if (!c.e4m3) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[row * c.dim + d]);
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(p[row * c.dim + d], __NV_E4M3))) * unit;
}

__global__ void __launch_bounds__(kWarps * 32) k_attn_decode(AttnArgs a) {
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][kMaxHeadDim];
  const int b = blockIdx.x / a.n_heads, h = blockIdx.x % a.n_heads;
  const CacheDev& c = a.cache;
  const int kv = h / (a.n_heads / c.heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_begin();
  int n = a.lens[b];
  const int64_t room = int64_t(a.table.max_pages) * c.page;
  if (n > room) {
    n = int(room);
    if (threadIdx.x == 0) report_bad_page(a.table.status_flags);
  }
  const int first = a.window > 0 ? max(0, n - a.window) : 0;
  constexpr int kPer = kMaxHeadDim / 32;
  float q[kPer], o[kPer] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < c.dim ? __bfloat162float(a.q[b * a.q_stride + h * c.dim + d]) : 0.0f;
  }
  for (int j = first + warp; j < n; j += kWarps) {
    const int page = a.table.pages[int64_t(b) * a.table.max_pages + j / c.page];
    if (page < 0 || page >= c.n_pages) {
      if (lane == 0) report_bad_page(a.table.status_flags);
      continue;
    }
    const int64_t row = (int64_t(page) * c.heads + kv) * c.page + j % c.page;
    const float ku = c.e4m3 ? exp_value(c.k_exp[row]) : 1.0f, vu = c.e4m3 ? exp_value(c.v_exp[row]) : 1.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < c.dim) s = fmaf(q[i], cache_value(c, c.k, row, lane + 32 * i, ku), s);
    const float t = warp_sum(s) * (a.scale * kLog2e);
    const float mn = fmaxf(m, t), base = mn == -INFINITY ? 0.0f : mn;
    const float p = exp2f(t - base), f = exp2f(m - base);
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < c.dim) o[i] = fmaf(p, cache_value(c, c.v, row, lane + 32 * i, vu), o[i] * f);
    m = mn;
  }
  if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
  for (int i = 0; i < kPer; ++i) sm_o[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float mt = -INFINITY, lt = 0.0f;
  for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm_m[w]);
  const float base = mt == -INFINITY ? 0.0f : mt;
  for (int w = 0; w < kWarps; ++w) lt += sm_l[w] * exp2f(sm_m[w] - base);
  for (int d = threadIdx.x; d < c.dim; d += blockDim.x) {
    float v = 0.0f;
    for (int w = 0; w < kWarps; ++w) v += sm_o[w][d] * exp2f(sm_m[w] - base);
    a.out[(int64_t(b) * a.n_heads + h) * c.dim + d] = __float2bfloat16(lt > 0.0f ? v / lt : 0.0f);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[int64_t(b) * a.n_heads + h] = lt > 0.0f ? base * kLn2 + logf(lt) : -INFINITY;
}

}  // namespace

size_t attn_workspace_bytes(const CacheDev&, int, int) { return kAttnPartialsAt; }

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s) {
  return launch_pdl(k_attn_decode, dim3(a.B * a.n_heads), dim3(kWarps * 32), 0, s, a);
}

}  // namespace moe
