// What stands between two blocks on the residual stream: the post-norm, gate and scale of a block's
// output, the residual sum, and the next block's norm, in one pass over [T, d].
//
// A CTA takes one row; a thread holds its part of the row in registers (kVecs groups of eight
// elements, the groups a CTA-width apart so that every access is a contiguous 16- or 32-byte one per
// thread), so y and the residual are read once and both results written once.  The two sums of
// squares are fp32: over a thread's elements, then the warp's lanes, then the warps in order (the
// result does not depend on scheduling).
#include "decoder.cuh"

namespace moe {
namespace {

// Sum over the CTA; `part` holds a value a warp.  Every thread gets the sum of the warps' sums in
// warp order.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < warps; ++i) s += part[i];
  return s;
}

__device__ __forceinline__ void load_any8(const void* p, bool bf16, int64_t i, float (&v)[8]) {
  if (bf16) load_vec8(static_cast<const __nv_bfloat16*>(p) + i, v);
  else load_vec8(static_cast<const float*>(p) + i, v);
}
__device__ __forceinline__ void store_any8(void* p, bool bf16, int64_t i, const float (&v)[8]) {
  if (bf16) store_vec8(static_cast<__nv_bfloat16*>(p) + i, v);
  else store_vec8(static_cast<float*>(p) + i, v);
}

template <int kVecs>
__global__ void __launch_bounds__(512) k_block_norm(NormArgs a) {
  __shared__ float part[2][16];
  const int64_t row0 = int64_t(blockIdx.x) * a.d;
  const int step = blockDim.x * 8;
  pdl_begin();
  float r[kVecs][8], z[kVecs][8];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int c = threadIdx.x * 8 + j * step;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[j][i] = z[j][i] = 0.0f;
    if (c < a.d) {
      load_any8(a.residual, a.r_bf16, row0 + c, r[j]);
      if (a.y) load_any8(a.y, a.y_bf16, row0 + c, z[j]);
    }
  }
  if (a.y) {
    float post = 1.0f;
    if (a.w_post) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += z[j][i] * z[j][i];
      post = rsqrtf(block_sum(s, part[0]) / float(a.d) + a.eps);
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int c = threadIdx.x * 8 + j * step;
      if (c >= a.d) continue;
      if (a.w_post) {
        float w[8];
        load_vec8(a.w_post + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[j][i] *= post * w[i];
      }
      if (a.gate) {
        float g[8];
        load_any8(a.gate, a.gate_bf16, int64_t(blockIdx.x) * a.gate_stride + c, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[j][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) r[j][i] = fmaf(a.alpha, z[j][i], r[j][i]);
    }
  }
  if (a.residual_out) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int c = threadIdx.x * 8 + j * step;
      if (c < a.d) store_any8(a.residual_out, a.r_bf16, row0 + c, r[j]);
    }
  }
  if (!a.x) return;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) s += r[j][i] * r[j][i];
  const float pre = rsqrtf(block_sum(s, part[1]) / float(a.d) + a.eps);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int c = threadIdx.x * 8 + j * step;
    if (c >= a.d) continue;
    float w[8];
    load_vec8(a.w_pre + c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] *= r[j][i] * pre;
    store_any8(a.x, a.x_bf16, row0 + c, w);
  }
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s) {
  // the fewest whole warps of eight elements a lane, up to 16 warps
  const int threads = std::min(512, (a.d / 8 + 31) / 32 * 32);
  const int vecs = (a.d + threads * 8 - 1) / (threads * 8);
  const dim3 grid(a.T), block(threads);
  if (vecs == 1) return launch_pdl(k_block_norm<1>, grid, block, 0, s, a);
  if (vecs == 2) return launch_pdl(k_block_norm<2>, grid, block, 0, s, a);
  return launch_pdl(k_block_norm<4>, grid, block, 0, s, a);
}

}  // namespace moe
