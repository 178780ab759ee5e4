// Microscaled 4-bit rows (include/mxfp4.h) on gfx950: what their kernels share.
//
// A row of C columns is padded to P, a multiple of 128.  Codes are e2m1 (sign, two exponent bits,
// one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), column 2j in the low half of byte j; every 32
// columns share a power of two, stored 127 above (255: NaN).
#pragma once

#include "common.h"
#include "launch.h"
#include "rows.h"

namespace w4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kMxBlock = 32;
constexpr int kFp4 = 4;  // the matrix instructions' operand format

// raw buffer resource (gfx9-class dword 3: 32-bit data format); loads past `bytes` read 0
__device__ __forceinline__ rsrc_t mx_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// The stored exponent of a block whose largest magnitude has these fp32 bits: its binary exponent
// less two, so that the magnitude in multiples of the power is in [4, 8).  Powers below 2^-127 (and
// subnormal magnitudes) get 2^-127; a block with an infinity or a NaN gets NaN.
__device__ __forceinline__ uint32_t mx_exponent(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 2;
  return amax_bits >= 0x7F800000u ? 255u : (uint32_t)(e > 0 ? e : 0);
}

// Its power of two in fp32 (2^-127 is subnormal there).
__device__ __forceinline__ float mx_power(uint32_t e) {
  return __uint_as_float(e == 255 ? 0x7FC00000u : e == 0 ? 0x00400000u : e << 23);
}

// Maximum over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_umax(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  return umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
}

// Eight columns of a row from column col, 0 past its last.
template <int DT>
__device__ __forceinline__ Raw8<DT> mx_chunk_of(const typename Elem<DT>::type* x, int col, int cols) {
  if (col + 8 <= cols) return load_raw8<DT>(x + col);
  return col < cols ? load_raw8_part<DT>(x + col, cols - col, 0u) : Raw8<DT>{};
}

// Codes of eight elements at power p, rounded to nearest even and held at 6 (the conversion takes
// the power off exactly, subnormal elements and powers included: checked over all 16-bit patterns
// at 14 powers and fp32 values at and beside every tie).
template <int DT>
__device__ __forceinline__ uint32_t mx_code8(const Raw8<DT>& r, float p) {
  uint32_t o = 0;
  if constexpr (DT == W4_DT_F32) {
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, __uint_as_float(r.q[0][0]), __uint_as_float(r.q[0][1]), p, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, __uint_as_float(r.q[0][2]), __uint_as_float(r.q[0][3]), p, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, __uint_as_float(r.q[1][0]), __uint_as_float(r.q[1][1]), p, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, __uint_as_float(r.q[1][2]), __uint_as_float(r.q[1][3]), p, 3);
  } else if constexpr (DT == W4_DT_F16) {
    const uint32_t w[4] = {r.q[0][0], r.q[0][1], r.q[0][2], r.q[0][3]};
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(o, __builtin_bit_cast(f16x2, w[0]), p, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(o, __builtin_bit_cast(f16x2, w[1]), p, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(o, __builtin_bit_cast(f16x2, w[2]), p, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(o, __builtin_bit_cast(f16x2, w[3]), p, 3);
  } else {
    const uint32_t w[4] = {r.q[0][0], r.q[0][1], r.q[0][2], r.q[0][3]};
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w[0]), p, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w[1]), p, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w[2]), p, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w[3]), p, 3);
  }
  return o;
}

// A chunk of eight columns, its quad of lanes holding the block of 32: codes, and the block's exponent.
template <int DT>
__device__ __forceinline__ uint32_t mx_chunk(const Raw8<DT>& r, uint32_t* exponent) {
  const uint32_t e = mx_exponent(quad_umax(absmax_bits<DT>(absmax8<DT>(r, 0u))));
  *exponent = e;
  return e == 255 ? 0u : mx_code8<DT>(r, mx_power(e));
}

// Byte B of word w (two codes) as a pair of bf16 times p, exactly (up to bf16's range).
template <int B>
__device__ __forceinline__ uint32_t mx_bf16x2(uint32_t w, float p) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, B));
}
__device__ __forceinline__ u32x4 mx_bf16x8(uint32_t w, float p) {
  return u32x4{mx_bf16x2<0>(w, p), mx_bf16x2<1>(w, p), mx_bf16x2<2>(w, p), mx_bf16x2<3>(w, p)};
}

__device__ __forceinline__ i32x8 mx_operand(const u32x4& v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

}  // namespace w4
