// What stands between two blocks on the residual stream: the post-norm, gate and scale of a block's
// output, the residual sum, and the next block's norm, in one pass over [T, d].
//
// A CTA takes a row at a time; a thread holds its part of the row in registers (kVecs groups of eight
// elements, the groups a CTA-width apart so that every access is a contiguous 16- or 32-byte one per
// thread), so y and the residual are read once and both results written once.  What bounds it is
// memory, and with more rows than CTAs fit on the GPU each CTA walks rows and loads its next one before
// it works on the current one, so that the two sums over the row, each a barrier, do not leave the
// memory idle (16384 rows of 2048 bf16: 44.8 us, 88 % of the measured copy rate; one row a CTA 62.6;
// two rows ahead 47.3).  The sums of squares are fp32: over a thread's elements, then the warp's lanes,
// then the warps in order (the result does not depend on scheduling).
#include "decoder.cuh"

namespace moe {
namespace {

// Sum over the CTA; `part` holds a value a warp, zeros behind them.  Every thread gets the sum of the
// warps' sums, added in one order.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < int(blockDim.x >> 5); i += 4) {
    const float4 p = *reinterpret_cast<const float4*>(part + i);
    s += (p.x + p.y) + (p.z + p.w);
  }
  return s;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Eight elements as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4& q = w[sizeof(T) == 2 ? 0 : i / 4];
      const int k = sizeof(T) == 2 ? i / 2 : i % 4;
      const uint32_t x = k == 0 ? q.x : k == 1 ? q.y : k == 2 ? q.z : q.w;
      v[i] = __uint_as_float(sizeof(T) == 4 ? x : i & 1 ? x & 0xffff0000u : x << 16);
    }
  }
};

// Threads that fit an SM: 64 registers hold one or two groups of eight with the next row's (with 42
// registers and 1536 threads the 16384 x 2048 case took 60.5 us against 46.1).
constexpr int kResident = 1024;

template <int kVecs, typename Y, typename R, typename X>
__global__ void __launch_bounds__(kResident, 1) k_block_norm(NormArgs a) {
  // of the two sums, alternating from row to row: one barrier a sum is enough
  __shared__ __align__(16) float part[4][kResident / 32];
  for (int i = threadIdx.x; i < 4 * kResident / 32; i += blockDim.x) part[0][i] = 0.0f;
  const int step = blockDim.x * 8, c0 = threadIdx.x * 8;
  const Y* y = static_cast<const Y*>(a.y);
  const R* residual = static_cast<const R*>(a.residual);
  __syncthreads();
  pdl_begin();
  Raw8<Y> y_next[kVecs];
  Raw8<R> r_next[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {  // zeros stay where a thread has no elements, or there is no y
    y_next[j].clear();
    r_next[j].clear();
  }
  auto fetch = [&](int row) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (c0 + j * step >= a.d) continue;
      const int64_t at = int64_t(row) * a.d + c0 + j * step;
      r_next[j].load(residual + at);
      if (y) y_next[j].load(y + at);
    }
  };
  // The next row's registers are for those that have them: two groups of fp32 would spill, and have the
  // next row brought to L2 instead (732 rows of 16384, fp32 y: 29.9 us against 32.3).
  constexpr bool kAhead = kVecs == 1 || sizeof(Y) + sizeof(R) == 4;
  if (kAhead) fetch(blockIdx.x);
  int turn = 0;
  for (int row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 2) {
    const int64_t row0 = int64_t(row) * a.d;
    const int next = row + gridDim.x;
    float r[kVecs][8], z[kVecs][8];
    if (!kAhead) fetch(row);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      r_next[j].unpack(r[j]);
      y_next[j].unpack(z[j]);
    }
    if (kAhead && next < a.T) fetch(next);
    if (!kAhead && next < a.T) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        if (c0 + j * step >= a.d) continue;
        const int64_t at = int64_t(next) * a.d + c0 + j * step;
        prefetch_l2(residual + at);
        if (y) prefetch_l2(y + at);
      }
    }
    if (y) {
      float scale = a.alpha;  // times the post-norm's 1 / rms
      if (a.w_post) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) s += z[j][i] * z[j][i];
        scale *= rsqrtf(fmaf(block_sum(s, part[turn]), a.inv_d, a.eps));
      }
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const int c = c0 + j * step;
        if (c >= a.d) continue;
        if (a.w_post) {
          float w[8];
          load_vec8(a.w_post + c, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[j][i] *= w[i];
        }
        if (a.gate) {
          float g[8];
          const int64_t at = int64_t(row) * a.gate_stride + c;
          if (a.gate_bf16) load_vec8(static_cast<const __nv_bfloat16*>(a.gate) + at, g);
          else load_vec8(static_cast<const float*>(a.gate) + at, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[j][i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) r[j][i] = fmaf(scale, z[j][i], r[j][i]);
      }
    }
    if (a.residual_out) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (c0 + j * step < a.d) store_vec8(static_cast<R*>(a.residual_out) + row0 + c0 + j * step, r[j]);
    }
    if (!a.x) continue;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += r[j][i] * r[j][i];
    const float pre = rsqrtf(fmaf(block_sum(s, part[turn + 1]), a.inv_d, a.eps));
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int c = c0 + j * step;
      if (c >= a.d) continue;
      float w[8];
      load_vec8(a.w_pre + c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] *= r[j][i] * pre;
      store_vec8(static_cast<X*>(a.x) + row0 + c, w);
    }
  }
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s) {
  // The fewest whole warps of eight elements a lane: fewer with more elements a lane are slower (8 -> 4
  // warps at 2048: 46.1 -> 47.7 us; 2 -> 1 at 512: 13.1 -> 13.9).  Past 4096 elements two CTAs of 16
  // warps with 16 elements a lane are better where both inputs are bf16 (1831 rows of 8192: 23.0 us, one
  // of 32 warps 27.6), one CTA of up to 32 with eight where one is fp32 (1464 rows: 24.9 against 28.8).
  const int most = a.y_bf16 && a.r_bf16 && a.d <= 8192 ? 512 : 1024;
  const int threads = std::min(most, (a.d / 8 + 31) / 32 * 32);
  auto by_type = [](bool bf16, auto f) { return bf16 ? f(__nv_bfloat16{}) : f(float{}); };
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  auto go = [&](auto v) {
    constexpr int kVecs = decltype(v)::value;
    const dim3 grid(std::min(a.T, sms * (kResident / threads)));
    return by_type(a.y_bf16, [&](auto y) {
      return by_type(a.r_bf16, [&](auto r) {
        return by_type(a.x_bf16, [&](auto x) {
          return launch_pdl(k_block_norm<kVecs, decltype(y), decltype(r), decltype(x)>, grid, dim3(threads), 0, s, a);
        });
      });
    });
  };
  return a.d <= threads * 8 ? go(std::integral_constant<int, 1>{}) : go(std::integral_constant<int, 2>{});
}

}  // namespace moe
