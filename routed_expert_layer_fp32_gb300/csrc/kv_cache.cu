// Writing keys and values into the paged cache (as bf16, or quantised to E4M3 with one power-of-two
// exponent a row) and reading them back.
//
// Both are copies bound by memory: a row is one token's key or value of one kv head.  A group of
// kLanes lanes takes the key and value rows of kHeadsEach heads of one token, eight elements a lane of
// each.  So the place in the cache, three dependent loads away (sequence and position, then page, then
// row), is looked up once for four rows, and four rows' loads are in flight together in every lane; a
// row's largest magnitude is a few shuffles.
//
// Exponent and codes: e is the smallest power with max|x| <= 448 * 2^e, taken from the maximum's
// bits.  x * 2^-e is exact (a power of two, and far from fp32's limits), so the code is the only
// rounding, and code * 2^e is exact in bf16 (4 significant bits): reading back adds none.
#include "decoder.cuh"

namespace moe {
namespace {

constexpr int kHeadsEach = 2;

// The row (an index over [n_pages, heads, page]) of token t and head 0 in the cache; -1 for a skipped
// or refused token.  Head h's row is h * page further.
__device__ __forceinline__ int64_t cache_row(const CacheDev& c, const PageTable& pt, const int32_t* seq,
                                             const int32_t* pos, int t) {
  const int p = __ldg(pos + t);
  const int s = seq ? __ldg(seq + t) : t;
  if (p < 0) return -1;
  const int slot = unsigned(p) / unsigned(c.page);
  int page = -1;
  if (s >= 0 && s < pt.n_seqs && slot < pt.max_pages) page = __ldg(pt.pages + int64_t(s) * pt.max_pages + slot);
  if (page < 0 || page >= c.n_pages) {
    report_bad_page(pt.status_flags);
    return -1;
  }
  return int64_t(page) * c.heads * c.page + (p - slot * c.page);
}

template <int kLanes>
__device__ __forceinline__ float group_max8(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float up) {
  uint2 c;
  c.x = uint32_t(e4m3_code2(x[0] * up, x[1] * up)) | uint32_t(e4m3_code2(x[2] * up, x[3] * up)) << 16;
  c.y = uint32_t(e4m3_code2(x[4] * up, x[5] * up)) | uint32_t(e4m3_code2(x[6] * up, x[7] * up)) << 16;
  return c;
}

template <int kLanes, bool kE4M3, typename Src>
__global__ void __launch_bounds__(256) k_kv_write(CacheDev c, PageTable pt, const Src* __restrict__ k,
                                                  const Src* __restrict__ v, int64_t k_stride, int64_t v_stride, int T,
                                                  const int32_t* __restrict__ seq, const int32_t* __restrict__ pos) {
  const int t = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int h0 = blockIdx.y * kHeadsEach, heads = min(kHeadsEach, c.heads - h0);
  const bool mine = t < T && lane * 8 < c.dim;
  pdl_begin();
  float kx[kHeadsEach][8], vx[kHeadsEach][8];
#pragma unroll
  for (int j = 0; j < kHeadsEach; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) kx[j][i] = vx[j][i] = 0.0f;
    if (mine && j < heads) {
      load_vec8(k + t * k_stride + (h0 + j) * c.dim + lane * 8, kx[j]);
      load_vec8(v + t * v_stride + (h0 + j) * c.dim + lane * 8, vx[j]);
    }
  }
  const int64_t row0 = t < T ? cache_row(c, pt, seq, pos, t) : -1;
#pragma unroll
  for (int j = 0; j < kHeadsEach; ++j) {
    const int64_t row = row0 + int64_t(h0 + j) * c.page;
    const bool write = row0 >= 0 && j < heads;
    if constexpr (kE4M3) {
      const uint32_t ke = row_exponent(group_max8<kLanes>(kx[j])), ve = row_exponent(group_max8<kLanes>(vx[j]));
      if (!write) continue;
      if (mine) {
        *reinterpret_cast<uint2*>(c.k + row * c.dim + lane * 8) = codes8(kx[j], inverse_exp_value(ke));
        *reinterpret_cast<uint2*>(c.v + row * c.dim + lane * 8) = codes8(vx[j], inverse_exp_value(ve));
      }
      if (lane == 0) c.k_exp[row] = uint8_t(ke);
      if (lane == 1) c.v_exp[row] = uint8_t(ve);
    } else {
      if (!write || !mine) continue;
      store_vec8(reinterpret_cast<__nv_bfloat16*>(c.k) + row * c.dim + lane * 8, kx[j]);
      store_vec8(reinterpret_cast<__nv_bfloat16*>(c.v) + row * c.dim + lane * 8, vx[j]);
    }
  }
}

// Eight codes times 2^e as fp32.
__device__ __forceinline__ void values8(uint2 codes, float unit, float (&v)[8]) {
  const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x * unit;
    v[2 * i + 1] = f.y * unit;
  }
}

template <int kLanes, bool kE4M3, typename Dst>
__global__ void __launch_bounds__(256) k_kv_read(CacheDev c, PageTable pt, int T, const int32_t* __restrict__ seq,
                                                 const int32_t* __restrict__ pos, Dst* __restrict__ k_out,
                                                 Dst* __restrict__ v_out) {
  const int t = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int h0 = blockIdx.y * kHeadsEach, heads = min(kHeadsEach, c.heads - h0);
  if (t >= T || lane * 8 >= c.dim) return;
  pdl_begin();
  const int64_t row0 = cache_row(c, pt, seq, pos, t);
  float kx[kHeadsEach][8], vx[kHeadsEach][8];
  uint2 kc[kHeadsEach], vc[kHeadsEach];
  uint32_t ke[kHeadsEach], ve[kHeadsEach];
#pragma unroll
  for (int j = 0; j < kHeadsEach; ++j) {
    const int64_t row = row0 + int64_t(h0 + j) * c.page;
    const bool read = row0 >= 0 && j < heads;
    if constexpr (kE4M3) {
      kc[j] = vc[j] = make_uint2(0u, 0u);  // zeros for a token that is not there
      ke[j] = ve[j] = kExpBias;
      if (read) {
        kc[j] = *reinterpret_cast<const uint2*>(c.k + row * c.dim + lane * 8);
        vc[j] = *reinterpret_cast<const uint2*>(c.v + row * c.dim + lane * 8);
        ke[j] = c.k_exp[row];
        ve[j] = c.v_exp[row];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) kx[j][i] = vx[j][i] = 0.0f;
      if (read) {
        load_vec8(reinterpret_cast<const __nv_bfloat16*>(c.k) + row * c.dim + lane * 8, kx[j]);
        load_vec8(reinterpret_cast<const __nv_bfloat16*>(c.v) + row * c.dim + lane * 8, vx[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kHeadsEach; ++j) {
    if (j >= heads) continue;
    if constexpr (kE4M3) {
      values8(kc[j], exp_value(ke[j]), kx[j]);
      values8(vc[j], exp_value(ve[j]), vx[j]);
    }
    const int64_t at = (int64_t(t) * c.heads + h0 + j) * c.dim + lane * 8;
    store_vec8(k_out + at, kx[j]);
    store_vec8(v_out + at, vx[j]);
  }
}

// The lanes of a row: a power of two that covers it with eight elements each.
template <typename F>
cudaError_t with_lanes(int dim, F f) {
  if (dim <= 64) return f(std::integral_constant<int, 8>{});
  if (dim <= 128) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

dim3 token_grid(int T, int lanes, int heads) {
  return dim3((T + 256 / lanes - 1) / (256 / lanes), (heads + kHeadsEach - 1) / kHeadsEach);
}

}  // namespace

cudaError_t launch_kv_write(const CacheDev& c, const PageTable& pt, const void* k, const void* v, bool bf16,
                            int64_t k_stride, int64_t v_stride, int T, const int32_t* seq, const int32_t* pos,
                            cudaStream_t s) {
  return with_lanes(c.dim, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const dim3 grid = token_grid(T, L, c.heads);
    auto go = [&](auto e4m3, auto src) {
      using Src = decltype(src);
      return launch_pdl(k_kv_write<L, decltype(e4m3)::value, Src>, grid, dim3(256), 0, s, c, pt,
                        static_cast<const Src*>(k), static_cast<const Src*>(v), k_stride, v_stride, T, seq, pos);
    };
    if (c.e4m3) return bf16 ? go(std::true_type{}, __nv_bfloat16{}) : go(std::true_type{}, float{});
    return bf16 ? go(std::false_type{}, __nv_bfloat16{}) : go(std::false_type{}, float{});
  });
}

cudaError_t launch_kv_read(const CacheDev& c, const PageTable& pt, int T, const int32_t* seq, const int32_t* pos,
                           void* k_out, void* v_out, bool bf16, cudaStream_t s) {
  return with_lanes(c.dim, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const dim3 grid = token_grid(T, L, c.heads);
    auto go = [&](auto e4m3, auto dst) {
      using Dst = decltype(dst);
      return launch_pdl(k_kv_read<L, decltype(e4m3)::value, Dst>, grid, dim3(256), 0, s, c, pt, T, seq, pos,
                        static_cast<Dst*>(k_out), static_cast<Dst*>(v_out));
    };
    if (c.e4m3) return bf16 ? go(std::true_type{}, __nv_bfloat16{}) : go(std::true_type{}, float{});
    return bf16 ? go(std::false_type{}, __nv_bfloat16{}) : go(std::false_type{}, float{});
  });
}

}  // namespace moe
