// Shared pieces of the decode-step operators: the paged key-value cache (kv_cache.cu, kv_rows.cuh), its pages
// (pages.cu), the rotary positions on the way into it (rope.cu), the attention that reads it (attn_decode.cu) and
// the norms between blocks (block_norm.cu).
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

// How a cache holds its rows.
enum class RowKind { kBf16, kE4M3, kInt4 };

// The cache as the kernels see it.
struct CacheDev {
  int n_pages, page, heads, dim;
  RowKind rows;
  uint8_t* k;  // rows of bf16, E4M3 or 4-bit codes
  uint8_t* v;
  uint8_t* k_exp;
  uint8_t* v_exp;
};
// And with what INT4 rows need besides.  The kernels of other rows are not given it: 16 bytes more of parameters made
// every call of the attention 0.1 to 0.3 us longer.
struct CacheScaled : CacheDev {
  uint8_t* k_scale;
  uint8_t* v_scale;
};
template <RowKind kRows>
using CacheOf = std::conditional_t<kRows == RowKind::kInt4, CacheScaled, CacheDev>;

// Bytes of a row's codes, and of its scales (INT4: whole words, so that they are read four at a time).
__host__ __device__ inline int row_bytes(RowKind rows, int dim) {
  return rows == RowKind::kBf16 ? 2 * dim : rows == RowKind::kE4M3 ? dim : dim / 2;
}
__host__ __device__ inline int scale_pitch(int dim) { return (dim + 63) / 64 * 4; }

// What other operators' kernels write (places, lengths, pages, queries, rows) is read by plain loads, in all of these
// files: the writer may still run when the reader's grid starts (pdl_begin), and a load through the read-only path (__ldg,
// or a const __restrict__ pointer) is for data that nobody writes while the grid lives.

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

// INT4 rows.  The stored exponents of rows of numbers, and of one with an infinity or a NaN in it.  At the
// low end the least scale, 2^-12 of the row's power, has to be a normal bf16 number; at the high end 192 times the
// largest a finite one (attn_decode.cu works with both).
constexpr int kInt4ExpLow = 16, kInt4ExpHigh = 246, kInt4ExpNaN = 255;
constexpr float kInt4Most = 7.0f;  // of the codes; times the largest scale: 105

// The stored exponent of a row whose largest magnitude is amax (finite): the smallest e with
// amax <= 105 * 2^e, from amax's bits (105 = 1.640625 * 2^6).
__device__ __forceinline__ uint32_t int4_row_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = int(u >> 23) - 6 + ((u & 0x7fffffu) > 0x520000u ? 1 : 0);
  return uint32_t(min(max(e, kInt4ExpLow), kInt4ExpHigh));
}

// The scale of byte b (0 .. 127): (1 + (b % 8) / 8) 2^(b / 8 - 12).
__device__ __forceinline__ float int4_scale(uint32_t b) { return __uint_as_float((b << 20) + (115u << 23)); }

// The smallest scale's byte with top <= 7 * scale (127 where there is none).  7 times a scale is exact, so that the
// comparisons decide, and the quotient's rounding does not.
__device__ __forceinline__ uint32_t int4_scale_byte(float top) {
  const float q = fmaxf(top * (1.0f / 7.0f), 0x1p-12f);
  uint32_t b = min(((__float_as_uint(q) + 0xfffffu) >> 20) - (115u << 3), 127u);
  if (b < 127u && kInt4Most * int4_scale(b) < top) ++b;
  else if (b > 0u && kInt4Most * int4_scale(b - 1u) >= top) --b;
  return b;
}

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

struct AttnScaledArgs : AttnArgs {  // of INT4 rows
  uint8_t* k_scale;
  uint8_t* v_scale;
};

size_t attn_workspace_bytes(const CacheDev& c, int n_heads, int B);
cudaError_t launch_attn_decode(const AttnScaledArgs& a, cudaStream_t s);
size_t attn_int4_workspace_bytes(const CacheDev& c, int n_heads);  // of these two, the part for INT4 caches
cudaError_t launch_attn_int4(const AttnScaledArgs& a, cudaStream_t s);

// Calls f with a constant: the lanes of a row (a power of two that covers it with eight elements each), the cache's
// kind of rows, or a value of the source's type.
template <typename F>
cudaError_t with_lanes(int dim, F f) {
  if (dim <= 64) return f(std::integral_constant<int, 8>{});
  if (dim <= 128) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}
template <typename F>
cudaError_t with_rows(RowKind rows, F f) {
  if (rows == RowKind::kE4M3) return f(std::integral_constant<RowKind, RowKind::kE4M3>{});
  if (rows == RowKind::kInt4) return f(std::integral_constant<RowKind, RowKind::kInt4>{});
  return f(std::integral_constant<RowKind, RowKind::kBf16>{});
}
template <typename F>
cudaError_t with_source(bool bf16, F f) {
  return bf16 ? f(__nv_bfloat16{}) : f(float{});
}

cudaError_t launch_kv_write(const CacheScaled& c, const PageTable& pt, const void* k, const void* v, bool bf16,
                            int64_t k_stride, int64_t v_stride, int T, const int32_t* seq, const int32_t* pos,
                            cudaStream_t s);
cudaError_t launch_kv_read(const CacheScaled& c, const PageTable& pt, int T, const int32_t* seq, const int32_t* pos,
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

// Pages of new tokens (pages.cu).  Workspace: the status record, then a word a sequence and one more.
constexpr int kMaxPagePositions = 1 << 28;
constexpr size_t kPagesWordsAt = sizeof(DevStatus);
inline size_t pages_workspace_bytes(int B) { return align_up(kPagesWordsAt + (size_t(B) + 1) * 4, 256); }

struct PlanArgs {
  const int32_t* lens;
  const int32_t* new_tokens;
  int B;
  int32_t* table;
  int max_pages;
  const int32_t* free_pages;
  const int32_t* n_free;
  int n_pages, page, max_tokens;
  int32_t *lens_out, *n_free_out, *starts, *seq, *pos, *slot;
  char* ws;
};
cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t s);

struct ReleaseArgs {
  const int32_t* lens;
  const uint8_t* ended;
  int B;
  const int32_t* table;
  int max_pages;
  int32_t* free_pages;
  const int32_t* n_free;
  int n_pages, page;
  int32_t *lens_out, *n_free_out;
  char* ws;
};
cudaError_t launch_page_release(const ReleaseArgs& a, cudaStream_t s);

// Rotary positions (rope.cu).
struct RopeDev {
  const uint64_t* turns;
  int dim;  // elements that are turned
  bool interleaved;
  float magnitude;
};
// Rows of heads of one tensor, `stride` elements from a token's to the next token's.
struct HeadRows {
  const void* x;
  int64_t stride;
  int heads;
};
struct RopeArgs {
  RopeDev rope;
  HeadRows q, k, v;  // k and v: heads 0 where there is no cache
  void* out;         // of q
  int64_t out_stride;
  CacheScaled cache;
  int dim, T;
  bool inverse;
  const int32_t* pos;
  const int32_t* slot;
  int* status_flags;
};
cudaError_t launch_rope(const RopeArgs& a, bool bf16, cudaStream_t s);           // out as x
cudaError_t launch_rope_kv_write(const RopeArgs& a, bool bf16, cudaStream_t s);  // out bf16, and the cache

}  // namespace moe
