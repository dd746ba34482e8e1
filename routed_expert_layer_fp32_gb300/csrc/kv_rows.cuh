// One row of the paged cache (a token's key or value of one kv head) from fp32 values and back, by a group of
// kLanes lanes with eight elements each.
//
// E4M3: e is the smallest power with max|x| <= 448 * 2^e, taken from the maximum's bits.  x * 2^-e is exact (a
// power of two, and far from fp32's limits), so the code is the only rounding, and code * 2^e is exact in bf16 (4
// significant bits): reading back adds none.
//
// INT4: e likewise with 105 (7 times the largest scale), then the smallest scale s of each 16 elements with
// 7 s >= max|x 2^-e|, then n = x 2^-e / s to the nearest whole number, ties to even.  The quotient is found by a
// reciprocal and put right by its remainder y - n s, which is exact in fp32 (n s is of 7 bits, and within a factor
// of two of y or 0): so n does not depend on how the reciprocal is rounded.  n s 2^e has 7 significant bits, and is
// exact in bf16 as well.
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

// y / s to the nearest whole number of -7 .. 7, ties to even, plus 8.
__device__ __forceinline__ uint32_t int4_code(float y, float s, float reciprocal) {
  float n = rintf(y * reciprocal);
  const float rest = fmaf(-n, s, y), over = fabsf(rest) - 0.5f * s;
  const float odd = fabsf(n - 2.0f * rintf(0.5f * n));  // 0 or 1
  if (over > 0.0f || (over == 0.0f && odd != 0.0f)) n += copysignf(1.0f, rest);
  n = fminf(fmaxf(n, -kInt4Most), kInt4Most);
  return __float_as_uint(n + (8388608.0f + 8.0f)) & 15u;  // 2^23: the whole number is in the low bits
}

// Four codes a half, as two 16-bit words turned left by 3.
__device__ __forceinline__ uint32_t int4_turned(uint32_t w) { return (w << 3 & 0xfff8fff8u) | (w >> 13 & 0x00070007u); }
__device__ __forceinline__ uint32_t int4_turned_back(uint32_t w) { return (w >> 3 & 0x1fff1fffu) | (w << 13 & 0xe000e000u); }

// Writes one row, if `write` holds (the same for the lanes of a group; all lanes of the warp come here).  x: the
// lane's eight elements, zeros past the row's end.
template <int kLanes, RowKind kRows>
__device__ __forceinline__ void store_row(const CacheDev& c, uint8_t* pool, uint8_t* exps, uint8_t* scales, int64_t row,
                                          bool write, int lane, const float (&x)[8]) {
  const bool mine = lane * 8 < c.dim;
  if constexpr (kRows == RowKind::kBf16) {
    if (write && mine) store_vec8(reinterpret_cast<__nv_bfloat16*>(pool) + row * c.dim + lane * 8, x);
  } else if constexpr (kRows == RowKind::kE4M3) {
    const uint32_t e = row_exponent(group_max8<kLanes>(x));
    if (!write) return;
    if (mine) *reinterpret_cast<uint2*>(pool + row * c.dim + lane * 8) = codes8(x, inverse_exp_value(e));
    if (lane == 0) exps[row] = uint8_t(e);
  } else {
    uint32_t top = 0;  // largest magnitude's bits: an infinity's or a NaN's are above all numbers'
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    uint32_t row_top = top;
#pragma unroll
    for (int o = kLanes / 2; o > 1; o >>= 1) row_top = max(row_top, __shfl_xor_sync(0xffffffffu, row_top, o));
    if (!write) return;
    const bool lost = row_top >= 0x7f800000u;
    const uint32_t e = lost ? uint32_t(kInt4ExpNaN) : int4_row_exponent(__uint_as_float(row_top));
    const float down = lost ? 0.0f : __uint_as_float((254u - e) << 23);  // 2^(127 - e)
    const uint32_t b = lost ? 127u : int4_scale_byte(__uint_as_float(top) * down);
    if (mine) {
      const float s = int4_scale(b), reciprocal = 1.0f / s;
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) w |= (lost ? 8u : int4_code(x[i] * down, s, reciprocal)) << (4 * i);
      reinterpret_cast<uint32_t*>(pool + row * (c.dim / 2))[lane] = int4_turned(w);
    }
    // a byte of two lanes; those past the row's end fill its last word with zeros
    const int pitch = scale_pitch(c.dim), at = lane >> 1;
    if ((lane & 1) == 0 && at < pitch) scales[row * pitch + at] = uint8_t(mine ? b : 0u);
    if (lane == 0) exps[row] = uint8_t(e);
  }
}

// One row's raw contents, loaded before they are needed (zeros for a row that is not there).
template <RowKind kRows>
struct RawRow {
  uint4 w;
  uint32_t exp, scale;
  __device__ __forceinline__ void load(const CacheDev& c, const uint8_t* pool, const uint8_t* exps, const uint8_t* scales,
                                       int64_t row, bool there, int lane) {
    w = make_uint4(0u, 0u, 0u, 0u);
    exp = kExpBias;
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
  __device__ __forceinline__ void values(bool there, float (&v)[8]) const {
    if constexpr (kRows == RowKind::kBf16) {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    } else if constexpr (kRows == RowKind::kE4M3) {
      values8(make_uint2(w.x, w.y), exp_value(exp), v);
    } else {
      const float unit = exp == kInt4ExpNaN ? __uint_as_float(0x7fc00000u)
                                            : there ? int4_scale(scale) * exp_value(exp) : 0.0f;
      const uint32_t u = int4_turned_back(w.x);
#pragma unroll
      for (int i = 0; i < 8; ++i)  // 2^23 + code
        v[i] = (__uint_as_float((u >> (4 * i) & 15u) | 0x4b000000u) - (8388608.0f + 8.0f)) * unit;
    }
  }
};

}  // namespace moe
