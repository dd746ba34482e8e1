// One row of the paged cache (a token's key or value of one kv head) from fp32 values and back, by a group of
// kLanes lanes with eight elements each.
//
// E4M3: e is the smallest power with max|x| <= 448 * 2^e, taken from the maximum's bits.  x * 2^-e is exact (a
// power of two, and far from fp32's limits), so the code is the only rounding, and code * 2^e is exact in bf16 (4
// significant bits): reading back adds none.
//
// INT4: e likewise with 105 (7 times the largest scale), then the smallest scale s of each 16 elements with
// 7 s >= max|x 2^-e|, then n = x 2^-e / s to the nearest whole number, ties to even.  n s 2^e has 7 significant
// bits, and is exact in bf16 as well.
#pragma once

#include "decoder.cuh"

namespace moe {

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

// Eight E4M3 codes times 2^e as fp32.
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

__constant__ const float kReciprocals[8] = {1.0f, 8.0f / 9, 8.0f / 10, 8.0f / 11, 8.0f / 12, 8.0f / 13, 8.0f / 14, 8.0f / 15};

// The largest of magnitudes, NaN where one of them is (fmaxf would leave it out).
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The codes of eight elements of magnitude up to 7 s, x_i / s to the nearest whole number, ties to even, plus 8, in the
// order of the cache (s the scale times the row's power of two, which changes no rounding here).  With the reciprocal rounded to
// nearest, the quotient put right by its remainder (exact, by a fused multiply-add) is the correctly rounded one
// [Markstein 1990]; and that lies on the same side of a border k + 1/2 as the exact one, or on it with it: a border
// times s has 7 bits, and the next fp32 number is further from it than the quotient's rounding reaches.  Added to
// 1.5 * 2^23 + 8 it is rounded to a whole number, whose code stands in the low bits; multiply-adds put the eight side by
// side, and what is above the low bits adds up to a constant.
__device__ __forceinline__ uint32_t int4_codes(const float (&x)[8], float s, float reciprocal) {
  constexpr float kWhole = 12582912.0f + 8.0f;
  constexpr uint32_t kAbove = 0x4b400000u;  // 1.5 * 2^23's bits
  uint32_t w = 0u - kAbove * 0x11111111u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = x[i] * reciprocal;
    const float n = fmaf(fmaf(-q, s, x[i]), reciprocal, q);
    w += __float_as_uint(n + kWhole) << (4 * i);
  }
  return (w << 3 & 0xfff8fff8u) | (w >> 13 & 0x00070007u);
}

// A word of codes taken apart: element i and i + 4 of its eight in the halves of r[i], as bf16 numbers times u, where
// u holds an eighth of the elements' unit (scale times the row's power of two) in both halves, and minus -192 u.  A code
// c = n + 8 at mantissa bits 3 to 6 of a bf16 number 128 makes it 192 + 8n, and one fused multiply-add gives 8n u without
// rounding (n u has 7 significant bits).  The cache's order of bits makes shifts unnecessary for four of the eight.
__device__ __forceinline__ uint32_t int4_fma(uint32_t x, uint32_t u, uint32_t minus) {
  const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&u),
                                   *reinterpret_cast<const __nv_bfloat162*>(&minus));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t int4_minus_192(uint32_t u) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u), __float2bfloat162_rn(-192.0f));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Codes 2j and 2j + 1 of both halves, as 192 + 8n; mask 0x00780078 and one 0x43004300.
__device__ __forceinline__ void int4_pair(uint32_t w, int j, uint32_t mask, uint32_t one, uint32_t& a, uint32_t& b) {
  if (j == 1) w = __byte_perm(w, 0u, 0x2301);  // each half's bytes exchanged: turned by 8
  const uint32_t x = w >> 4;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(a) : "r"(w), "r"(mask), "r"(one));  // (w & mask) | one
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(b) : "r"(x), "r"(mask), "r"(one));
}
// u of a scale byte and an exponent byte: the scale's three mantissa bits and four exponent bits moved to their places,
// and the exponents added, all biased.  kInt4Zero with scale byte 0 gives u = 0, whatever the codes are; exponent 255 with
// scale 127 a NaN, and then so are the values.
constexpr uint32_t kInt4Zero = 15;
__device__ __forceinline__ uint32_t int4_unit(uint32_t scale, uint32_t exp) {
  return (scale * 16u + (exp - kInt4Zero) * 128u) * 0x00010001u;
}

// How a row is held: found by all lanes of its group together, then written by them.  x: the lane's eight elements, zeros
// past the row's end.
template <RowKind kRows>
struct RowCode {
  uint32_t exp, scale;  // of the row, and (INT4) of the lane's sixteen elements
  template <int kLanes>
  __device__ __forceinline__ void find(const float (&x)[8]) {
    if constexpr (kRows == RowKind::kE4M3) exp = row_exponent(group_max8<kLanes>(x));
    if constexpr (kRows == RowKind::kInt4) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max_or_nan(top, fabsf(x[i]));
      top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
      float row_top = top;
#pragma unroll
      for (int o = kLanes / 2; o > 1; o >>= 1) row_top = max_or_nan(row_top, __shfl_xor_sync(0xffffffffu, row_top, o));
      const bool lost = !(row_top < INFINITY);
      exp = lost ? uint32_t(kInt4ExpNaN) : int4_row_exponent(row_top);
      scale = lost ? 127u : int4_scale_byte(top * __uint_as_float((254u - exp) << 23));  // times 2^(127 - exp)
    }
  }
  // exp_lane: who writes the exponent
  __device__ __forceinline__ void store(const CacheOf<kRows>& c, uint8_t* pool, uint8_t* exps, uint8_t* scales, int64_t row,
                                        int lane, int exp_lane, float (&x)[8]) const {
    const bool mine = lane * 8 < c.dim;
    if constexpr (kRows == RowKind::kBf16) {
      if (mine) store_vec8(reinterpret_cast<__nv_bfloat16*>(pool) + row * c.dim + lane * 8, x);
      return;
    }
    if constexpr (kRows == RowKind::kE4M3) {
      if (mine) *reinterpret_cast<uint2*>(pool + row * c.dim + lane * 8) = codes8(x, inverse_exp_value(exp));
    }
    if constexpr (kRows == RowKind::kInt4) {
      if (mine) {
        const float s = int4_scale(scale) * __uint_as_float(exp << 23);
        // of the eight mantissas a scale has, each rounded to nearest, times powers of two
        const float reciprocal = kReciprocals[scale & 7] * (__uint_as_float((139u - (scale >> 3)) << 23) *
                                                            __uint_as_float((254u - exp) << 23));
        if (__builtin_expect(exp == kInt4ExpHigh, 0)) {  // magnitudes past 7 s
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -kInt4Most * s), kInt4Most * s);
        }
        reinterpret_cast<uint32_t*>(pool + row * (c.dim / 2))[lane] = int4_codes(x, s, reciprocal);
      }
      // a byte of two lanes; those past the row's end fill its last word with zeros
      const int pitch = scale_pitch(c.dim), at = lane >> 1;
      if ((lane & 1) == 0 && at < pitch) scales[row * pitch + at] = uint8_t(mine ? scale : 0u);
    }
    if (lane == exp_lane) exps[row] = uint8_t(exp);
  }
};

// The scales of keys and values where there are any.
template <RowKind kRows>
__device__ __forceinline__ uint8_t* scales_of(const CacheOf<kRows>& c, bool keys) {
  if constexpr (kRows == RowKind::kInt4) return keys ? c.k_scale : c.v_scale;
  else return nullptr;
}

// One row's raw contents, loaded before they are needed (zeros for a row that is not there).
template <RowKind kRows>
struct RawRow {
  uint4 w;
  uint32_t exp, scale;
  __device__ __forceinline__ void load(const CacheOf<kRows>& c, const uint8_t* pool, const uint8_t* exps, const uint8_t* scales,
                                       int64_t row, bool there, int lane) {
    w = make_uint4(0u, 0u, 0u, 0u);
    exp = kRows == RowKind::kInt4 ? kInt4Zero : kExpBias;
    scale = 0u;
    if (!there) return;
    if constexpr (kRows == RowKind::kBf16) {
      w = *reinterpret_cast<const uint4*>(pool + (row * c.dim + lane * 8) * 2);
    } else if constexpr (kRows == RowKind::kE4M3) {
      const uint2 u = *reinterpret_cast<const uint2*>(pool + row * c.dim + lane * 8);
      w.x = u.x, w.y = u.y;
      exp = exps[row];
    } else {
      w.x = reinterpret_cast<const uint32_t*>(pool + row * (c.dim / 2))[lane];
      exp = exps[row];
      scale = scales[row * scale_pitch(c.dim) + (lane >> 1)];
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (kRows == RowKind::kE4M3) {
      values8(make_uint2(w.x, w.y), exp_value(exp), v);
      return;
    }
    if constexpr (kRows == RowKind::kInt4) bf16x8(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  }
  // INT4: the eight elements in bf16, which holds them exactly.
  __device__ __forceinline__ void bf16x8(uint32_t (&u)[4]) const {
    const uint32_t unit = int4_unit(scale, exp), minus = int4_minus_192(unit);
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      int4_pair(w.x, j, 0x00780078u, 0x43004300u, r[2 * j], r[2 * j + 1]);
      r[2 * j] = int4_fma(r[2 * j], unit, minus);
      r[2 * j + 1] = int4_fma(r[2 * j + 1], unit, minus);
    }
    u[0] = __byte_perm(r[0], r[1], 0x5410);
    u[1] = __byte_perm(r[2], r[3], 0x5410);
    u[2] = __byte_perm(r[0], r[1], 0x7632);
    u[3] = __byte_perm(r[2], r[3], 0x7632);
  }
  __device__ __forceinline__ void store(float* p) const {
    float v[8];
    values(v);
    store_vec8(p, v);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    if constexpr (kRows == RowKind::kE4M3) {
      float v[8];
      values(v);
      store_vec8(p, v);
    } else {
      uint32_t u[4] = {w.x, w.y, w.z, w.w};
      if constexpr (kRows == RowKind::kInt4) bf16x8(u);
      *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
};

}  // namespace moe
