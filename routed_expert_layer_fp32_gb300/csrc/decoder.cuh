// Shared pieces of the decode-step operators: the paged key-value cache (kv_cache.cu), the
// attention that reads it (attn_decode.cu) and the norms between blocks (block_norm.cu).
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "per_device.cuh"

namespace moe {

constexpr int kMaxPageSize = 4096;
constexpr int kMaxHeadDim = 256;
constexpr int kMaxHeads = 1024;
constexpr int kMaxSeqs = 1 << 16;
constexpr int kMaxNormDim = 16384;
constexpr int kExpBias = 127;  // of the stored row exponents

// The cache as the kernels see it.
struct CacheDev {
  int n_pages, page, heads, dim;
  bool e4m3;
  uint8_t* k;  // bf16 or E4M3 rows
  uint8_t* v;
  uint8_t* k_exp;
  uint8_t* v_exp;
};

// A page table on the device and where its violations are recorded.
struct PageTable {
  const int32_t* pages;
  int n_seqs, max_pages;
  int* status_flags;
};

__device__ __forceinline__ void report_bad_page(int* status_flags) { atomicOr(status_flags, kFlagBadPage); }

// 2^(exp - 127) for a stored exponent: normal from 1 on, and the subnormal 2^-127 for 0.
__device__ __forceinline__ float exp_value(uint32_t exp) { return __uint_as_float(exp ? exp << 23 : 0x00400000u); }

// The stored exponent of a row whose largest magnitude is amax: the smallest e >= -127 with
// amax <= 448 * 2^e, from amax's bits (448 = 1.75 * 2^8), biased by 127.  An infinite amax gives
// the exponent of 2^128.
__device__ __forceinline__ uint32_t row_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = int(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return uint32_t(max(e, -kExpBias) + kExpBias);
}

// 2^(127 - exp), exact for every exponent row_exponent gives (0 .. 247).
__device__ __forceinline__ float inverse_exp_value(uint32_t exp) { return __uint_as_float((254u - exp) << 23); }

// Eight consecutive elements as fp32; p 16-byte aligned.
__device__ __forceinline__ void load_vec8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load_vec8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void store_vec8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store_vec8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

inline int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

inline int sm_count() {
  static std::atomic<int> kept[kMaxDevices];
  const int dev = current_device();
  return once_a_device(kept, dev, [dev] {
    int n = 0;
    return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
  });
}

// Workspace of the attention: the status record, then the join counters and partial results of
// attn_decode.cu.
constexpr size_t kAttnTicketsAt = sizeof(DevStatus);
constexpr int kAttnTickets = 1024;  // an upper bound of the attention grid
constexpr size_t kAttnPartialsAt = kAttnTicketsAt + size_t(kAttnTickets) * 4;

struct AttnArgs {
  CacheDev cache;
  PageTable table;
  const __nv_bfloat16* q;
  int64_t q_stride;
  int n_heads, B, window;
  float scale;
  const int32_t* lens;
  __nv_bfloat16* out;
  float* lse;
  char* ws;
};

size_t attn_workspace_bytes(const CacheDev& c, int n_heads, int B);
cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_kv_write(const CacheDev& c, const PageTable& pt, const void* k, const void* v, bool bf16,
                            int64_t k_stride, int64_t v_stride, int T, const int32_t* seq, const int32_t* pos,
                            cudaStream_t s);
cudaError_t launch_kv_read(const CacheDev& c, const PageTable& pt, int T, const int32_t* seq, const int32_t* pos,
                           void* k_out, void* v_out, bool bf16, cudaStream_t s);

struct NormArgs {
  const void* y;
  const float* w_post;
  const void* gate;
  int64_t gate_stride;
  float alpha, eps, inv_d;
  const void* residual;
  void* residual_out;
  const float* w_pre;
  void* x;
  bool y_bf16, gate_bf16, r_bf16, x_bf16;
  int T, d;
};
cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s);

}  // namespace moe
