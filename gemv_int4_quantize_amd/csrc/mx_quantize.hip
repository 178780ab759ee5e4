// Rows to microscaled 4-bit rows and back (mx4_quantize_rows, mx4_dequantize_rows), and float rows
// to bf16 parts, for gfx950.  All three are streams, bound by memory: a lane takes eight columns,
// and the four lanes of a quad a block of 32, whose largest magnitude they share by two exchanges, so
// that X is read once.  11008 x 4096 bf16 (90 MB of floats, 24 of rows): quantized in 20.5 us (5.6 TB/s
// of reads and writes together), back in 18.0 (6.3); a library copy reaches 5.1.  Few rows take a launch:
// 64 x 4096 2.6 us.
#include <algorithm>

#include "api_common.h"
#include "mx.h"

namespace w4 {

namespace {

constexpr int kChunks = 2;  // of eight columns, that a lane has in flight (4: 64 rows of 4096 3.4 us instead of 2.8)

// Chunk i of [rows][pc] chunks: its row and its place in it.  i counts from a row's start (base).
struct Place {
  int64_t row;
  int chunk;
};
__device__ __forceinline__ Place place(int64_t base_row, uint32_t in_row, uint32_t ahead, uint32_t pc) {
  const uint32_t at = in_row + ahead, rows = at / pc;
  return Place{base_row + rows, (int)(at - rows * pc)};
}

template <int DT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ X, int64_t rows, int cols, int64_t ld,
                                                          int pc, uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const typename Elem<DT>::type* x = static_cast<const typename Elem<DT>::type*>(X);
  const int64_t first = (int64_t)blockIdx.x * (256 * kChunks);
  const int64_t row0 = first / pc;
  const uint32_t in_row = (uint32_t)(first - row0 * pc);
  Raw8<DT> r[kChunks];
  Place at[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    at[c] = place(row0, in_row, c * 256 + threadIdx.x, (uint32_t)pc);
    r[c] = Raw8<DT>{};
    if (at[c].row < rows) r[c] = mx_chunk_of<DT>(x + at[c].row * ld, at[c].chunk * 8, cols);
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    uint32_t e;
    const uint32_t w = mx_chunk<DT>(r[c], &e);
    if (at[c].row >= rows) continue;
    const int64_t i = at[c].row * pc + at[c].chunk;
    *reinterpret_cast<uint32_t*>(codes + i * 4) = w;
    if ((at[c].chunk & 3) == 0) scales[i >> 2] = (uint8_t)e;
  }
}

// Eight columns of one row from codes: fp32, or rounded to fp16 / bf16 (bf16 holds them exactly).
template <int DT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t rows, int cols,
                                                            int pc, void* __restrict__ out, int64_t ldo) {
  typedef typename Elem<DT>::type E;
  typedef typename Elem<DT>::loose loose;
  const int64_t first = (int64_t)blockIdx.x * (256 * kChunks);
  const int64_t row0 = first / pc;
  const uint32_t in_row = (uint32_t)(first - row0 * pc);
  uint32_t w[kChunks], e[kChunks];
  Place at[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    at[c] = place(row0, in_row, c * 256 + threadIdx.x, (uint32_t)pc);
    w[c] = e[c] = 0;
    if (at[c].row >= rows || at[c].chunk * 8 >= cols) continue;
    const int64_t i = at[c].row * pc + at[c].chunk;
    w[c] = *reinterpret_cast<const uint32_t*>(codes + i * 4);
    e[c] = scales[i >> 2];
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = at[c].chunk * 8;
    if (at[c].row >= rows || col >= cols) continue;
    const float p = mx_power(e[c]);
    E* o = static_cast<E*>(out) + at[c].row * ldo + col;
    u32x4 q[DT == W4_DT_F32 ? 2 : 1];
    if constexpr (DT == W4_DT_BF16) {
      q[0] = mx_bf16x8(w[c], p);
    } else {
      f32x2 v[4];
      v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c], p, 0);
      v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c], p, 1);
      v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c], p, 2);
      v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c], p, 3);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DT == W4_DT_F32) {
          q[j >> 1][2 * (j & 1)] = __float_as_uint(v[j][0]);
          q[j >> 1][2 * (j & 1) + 1] = __float_as_uint(v[j][1]);
        } else {
          q[0][j] = pack_f16x2(v[j][0], v[j][1]);
        }
      }
    }
    if (col + 8 <= cols) {
      *reinterpret_cast<loose*>(o) = q[0];
      if constexpr (DT == W4_DT_F32) *reinterpret_cast<loose*>(o + 4) = q[1];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (col + j >= cols) break;
        if constexpr (DT == W4_DT_F32) o[j] = __uint_as_float(q[j >> 2][j & 3]);
        else o[j] = (uint16_t)(q[0][j >> 1] >> (16 * (j & 1)));
      }
    }
  }
}

// Rows as NP bf16 parts whose sum they are: out [rows][NP][pitch], zeros past the last column.  Each
// part is the rest cut to bf16 (toward zero, so that none overflows): eight bits of it, so that two
// parts hold an fp16 and three an fp32 (down to bf16's least number, 2^-133).  An infinity or a NaN
// is one in the first part and 0 in the others.
template <int DT, int NP>
__global__ __launch_bounds__(256) void mx_parts_kernel(const void* __restrict__ X, int64_t rows, int cols, int64_t ld, int pc,
                                                       uint16_t* __restrict__ out) {
  const typename Elem<DT>::type* x = static_cast<const typename Elem<DT>::type*>(X);
  const int64_t first = (int64_t)blockIdx.x * 256;
  const int64_t row0 = first / pc;
  const Place at = place(row0, (uint32_t)(first - row0 * pc), threadIdx.x, (uint32_t)pc);
  if (at.row >= rows) return;
  const Raw8<DT> r = mx_chunk_of<DT>(x + at.row * ld, at.chunk * 8, cols);
  uint16_t* o = out + (at.row * NP * pc + at.chunk) * 8;
  if constexpr (NP == 1) {
    *reinterpret_cast<u32x4*>(o) = r.q[0];
  } else {
    float v[8];
    widen8<DT>(r, v);
    const float whole[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      u32x4 q;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const float f = v[2 * j + s];
          const bool odd = (__float_as_uint(whole[2 * j + s]) & 0x7FFFFFFFu) >= 0x7F800000u;
          h[s] = __float_as_uint(f) >> 16;
          if (odd) h[s] = p > 0 ? 0u : (__float_as_uint(f) & 0x7FFFFFu) != 0 ? 0x7FC0u : h[s];
          v[2 * j + s] = f - __uint_as_float(h[s] << 16);
        }
        q[j] = h[0] | h[1] << 16;
      }
      *reinterpret_cast<u32x4*>(o + (int64_t)p * pc * 8) = q;
    }
  }
}

// Launches of at most 2^30 chunks: fewer than 2^32 threads, and 32-bit places within a block.
template <typename F>
hipError_t in_runs(int64_t rows, int64_t pc, F f) {
  const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 30) / pc);
  for (int64_t r = 0; r < rows; r += most) {
    f(r, std::min(most, rows - r));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t quantize(const void* X, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const int64_t pc = mx_pitch(cols) / 8;
  return in_runs(rows, pc, [&](int64_t r, int64_t n) {
    mx_quantize_kernel<DT><<<(unsigned)((n * pc + 256 * kChunks - 1) / (256 * kChunks)), 256, 0, st>>>(
        static_cast<const typename Elem<DT>::type*>(X) + r * ld, n, (int)cols, ld, (int)pc, codes + r * pc * 4,
        scales + r * pc / 4);
  });
}

template <int DT>
hipError_t dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out, int64_t ldo,
                      hipStream_t st) {
  const int64_t pc = mx_pitch(cols) / 8;
  return in_runs(rows, pc, [&](int64_t r, int64_t n) {
    mx_dequantize_kernel<DT><<<(unsigned)((n * pc + 256 * kChunks - 1) / (256 * kChunks)), 256, 0, st>>>(
        codes + r * pc * 4, scales + r * pc / 4, n, (int)cols, (int)pc,
        static_cast<typename Elem<DT>::type*>(out) + r * ldo, ldo);
  });
}

template <int DT, int NP>
hipError_t parts(const void* X, int64_t rows, int64_t cols, int64_t ld, int64_t pitch, uint16_t* out, hipStream_t st) {
  const int64_t pc = pitch / 8;
  return in_runs(rows, pc, [&](int64_t r, int64_t n) {
    mx_parts_kernel<DT, NP><<<(unsigned)((n * pc + 255) / 256), 256, 0, st>>>(
        static_cast<const typename Elem<DT>::type*>(X) + r * ld, n, (int)cols, ld, (int)pc, out + r * NP * pitch);
  });
}

}  // namespace

hipError_t launch_mx_quantize(const void* X, int dt, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                              uint8_t* scales, hipStream_t st) {
  switch (dt) {
    case W4_DT_F32: return quantize<W4_DT_F32>(X, rows, cols, ld, codes, scales, st);
    case W4_DT_F16: return quantize<W4_DT_F16>(X, rows, cols, ld, codes, scales, st);
    default: return quantize<W4_DT_BF16>(X, rows, cols, ld, codes, scales, st);
  }
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out, int dt,
                                int64_t ldo, hipStream_t st) {
  switch (dt) {
    case W4_DT_F32: return dequantize<W4_DT_F32>(codes, scales, rows, cols, out, ldo, st);
    case W4_DT_F16: return dequantize<W4_DT_F16>(codes, scales, rows, cols, out, ldo, st);
    default: return dequantize<W4_DT_BF16>(codes, scales, rows, cols, out, ldo, st);
  }
}

hipError_t launch_mx_parts(const void* X, int dt, int64_t rows, int64_t cols, int64_t ld, int64_t pitch, uint16_t* out,
                           hipStream_t st) {
  switch (dt) {
    case W4_DT_F32: return parts<W4_DT_F32, 3>(X, rows, cols, ld, pitch, out, st);
    case W4_DT_F16: return parts<W4_DT_F16, 2>(X, rows, cols, ld, pitch, out, st);
    default: return parts<W4_DT_BF16, 1>(X, rows, cols, ld, pitch, out, st);
  }
}

}  // namespace w4
