// Element loads of rows that need not be aligned to more than their element.
#pragma once

#include "common.h"
#include "launch.h"

namespace w4 {

typedef u32x4 u32x4_by2 __attribute__((aligned(2)));
typedef u32x4 u32x4_by4 __attribute__((aligned(4)));

template <int DT>
struct Elem {
  typedef uint16_t type;
  typedef u32x4_by2 loose;  // 16 bytes at an element's alignment
};
template <>
struct Elem<W4_DT_F32> {
  typedef float type;
  typedef u32x4_by4 loose;
};

// Eight elements as loaded: one 16-byte load (two for fp32), from an address that is
// aligned to the element only (gfx950 takes such addresses in one request).
template <int DT>
struct Raw8 {
  u32x4 q[DT == W4_DT_F32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const typename Elem<DT>::type* p) {
  typedef typename Elem<DT>::loose loose;
  Raw8<DT> r;
  r.q[0] = *reinterpret_cast<const loose*>(p);
  if constexpr (DT == W4_DT_F32) r.q[1] = *reinterpret_cast<const loose*>(p + 4);
  return r;
}

// The first n (< 8) of eight elements, the rest as `fill` bits.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8_part(const typename Elem<DT>::type* p, int n, uint32_t fill) {
  Raw8<DT> r;
  if constexpr (DT == W4_DT_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.q[j >> 2][j & 3] = j < n ? __float_as_uint(p[j]) : fill;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = 2 * j < n ? p[2 * j] : fill, hi = 2 * j + 1 < n ? p[2 * j + 1] : fill;
      r.q[0][j] = lo | hi << 16;
    }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& r, float v[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (DT == W4_DT_F32) v[j] = __uint_as_float(r.q[j >> 2][j & 3]);
    else if constexpr (DT == W4_DT_F16) v[j] = f16_bits_to_f32((r.q[0][j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
    else v[j] = __uint_as_float(j & 1 ? r.q[0][j >> 1] & 0xFFFF0000u : r.q[0][j >> 1] << 16);
  }
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Maximum over the wave in every lane, without LDS round trips: partners lane ^ 32 and ^ 16
// by permlane swaps, then row mirror, half-row mirror and quad permutes.
__device__ __forceinline__ float wave_max(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false)));
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false)));
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false)));
  return __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false)));
}

// wave_max of unsigned integers.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = umax(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = umax(b[0], b[1]);
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  return umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
}

template <int DT>
__device__ __forceinline__ float elem_to_f32(typename Elem<DT>::type x) {
  if constexpr (DT == W4_DT_F32) return x;
  else if constexpr (DT == W4_DT_F16) return f16_bits_to_f32(x);
  else return bf16_bits_to_f32(x);
}

// Row quantization to int8 (w8_quantize_rows).  The largest magnitude is kept as the bits of
// |x|, compared as integers: they order finite values, then infinity, then NaN.  16-bit types
// are compared as they are, two at a time (v_pk_max_u16); absmax_bits gives the maximum as fp32
// bits.
template <int DT>
__device__ __forceinline__ uint32_t absmax8(const Raw8<DT>& r, uint32_t m) {
  if constexpr (DT == W4_DT_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = umax(m, r.q[j >> 2][j & 3] & 0x7FFFFFFFu);
    return m;
  } else {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 v = __builtin_bit_cast(u16x2, m);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v = __builtin_elementwise_max(v, __builtin_bit_cast(u16x2, r.q[0][j] & 0x7FFF7FFFu));
    return __builtin_bit_cast(uint32_t, v);
  }
}

template <int DT>
__device__ __forceinline__ uint32_t absmax_bits(uint32_t m) {
  if constexpr (DT == W4_DT_F32) return m;
  const uint32_t b = umax(m & 0xFFFFu, m >> 16);
  if constexpr (DT == W4_DT_BF16) return b << 16;
  else return __float_as_uint(f16_bits_to_f32(b));
}

struct RowScale {
  float s, inv;
};

// Scale and reciprocal of a row from its absmax bits; both divisions are IEEE.  A row with
// an infinity or a NaN gets s = NaN and inv = 0 (code8 turns what is not finite to 0).
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale r;
  if (amax_bits >= 0x7F800000u) {
    r.s = __uint_as_float(0x7FC00000u);
    r.inv = 0.0f;
    return r;
  }
  const float s = __uint_as_float(amax_bits) / 127.0f;
  r.s = s > 0x1p-126f ? s : 0x1p-126f;
  r.inv = 1.0f / r.s;
  return r;
}

// rint(fp32(x * inv)) as a two's complement byte in the low bits: |x * inv| <= 127 (plus an
// ulp), so adding 1.5 * 2^23 rounds it to an integer, ties to even, in the low mantissa bits.
// The product is rounded by itself first (no contraction with the add).
__device__ __forceinline__ uint32_t code_bits(float x, float inv) {
#pragma clang fp contract(off)
  const float p = x * inv;
  return __float_as_uint(p + 12582912.0f);
}

// One output value of the int8 product before its bias: two rounded products, never
// contracted, so that every kernel gives the same bits.  The channel's scale comes first:
// sum * channel scale stays in range for any sensible weight, so the last product (by a
// token's scale of any size) overflows only where the result itself does.
__device__ __forceinline__ float w8_scaled(int acc, float sa, float sw) {
#pragma clang fp contract(off)
  const float p = (float)acc * sw;
  return p * sa;
}

template <int DT>
__device__ __forceinline__ u32x2 code8(const Raw8<DT>& r, float inv) {
  float v[8];
  widen8<DT>(r, v);
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = code_bits(v[j], inv);
  // bytes 0 of b[0..3] -> one word: two byte permutes and a merge
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000C0Cu);
    o[h] = lo | hi;
  }
  return o;
}

}  // namespace w4
