// Rows to int8 codes with one fp32 scale a row (w8_quantize_rows), for gfx950:
//   a = max |x|,  s = max(a / 127, 2^-126),  q = rint(x * fp32(1 / s)).
// An HBM stream that needs the whole row's maximum before its first code: a row is held in
// the registers of TPR threads (C chunks of eight elements each), so it is read once.
// Measured: bf16 [4096][4096] 10.4 us, 4.8 TB/s of 4.7 that a large copy reaches; 32 rows of
// 11008 3.8 us, little above a launch's least time.
#include <algorithm>

#include "api_common.h"
#include "launch.h"
#include "rows.h"

namespace w4 {

namespace {

template <int DT, int TPR, int C>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void quantize_rows_kernel(const void* __restrict__ X, int64_t rows,
                                                                               int cols, int64_t ld, int pitch,
                                                                               int8_t* __restrict__ codes,
                                                                               float* __restrict__ scales) {
  typedef typename Elem<DT>::type T;
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  constexpr int RPB = BLOCK / TPR;  // rows per block
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < rows;
  const T* x = static_cast<const T*>(X) + (live ? row : 0) * ld;
  Raw8<DT> r[C];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * TPR + t) * 8;
    if (live && col + 8 <= cols) r[c] = load_raw8<DT>(x + col);
    else if (live && col < cols) r[c] = load_raw8_part<DT>(x + col, cols - col, 0u);
    else r[c] = Raw8<DT>{};
  }
#pragma unroll
  for (int c = 0; c < C; ++c) m = absmax8<DT>(r[c], m);
  m = wave_umax(absmax_bits<DT>(m));
  if constexpr (TPR > 64) {
    __shared__ uint32_t part[TPR / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) m = part[i] > m ? part[i] : m;
  }
  if (!live) return;
  const RowScale rs = row_scale(m);
  const bool bad = m >= 0x7F800000u;
  if (t == 0) scales[row] = rs.s;
  int8_t* q = codes + row * pitch;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * TPR + t) * 8;
    if (col >= pitch) continue;
    const u32x2 o = bad ? u32x2{0u, 0u} : code8<DT>(r[c], rs.inv);
    *reinterpret_cast<u32x2*>(q + col) = o;
  }
}

// Rows too long for registers: one block a row, read twice (the second time from cache
// where it fits).
template <int DT>
__global__ __launch_bounds__(1024) void quantize_long_rows_kernel(const void* __restrict__ X, int cols, int64_t ld,
                                                                  int pitch, int8_t* __restrict__ codes,
                                                                  float* __restrict__ scales) {
  typedef typename Elem<DT>::type T;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(X) + row * ld;
  auto load = [&](int col) {
    if (col + 8 <= cols) return load_raw8<DT>(x + col);
    return col < cols ? load_raw8_part<DT>(x + col, cols - col, 0u) : Raw8<DT>{};
  };
  uint32_t m = 0;
  for (int col = threadIdx.x * 8; col < cols; col += 8192) m = absmax8<DT>(load(col), m);
  m = wave_umax(absmax_bits<DT>(m));
  __shared__ uint32_t part[16];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) m = part[i] > m ? part[i] : m;
  const RowScale rs = row_scale(m);
  const bool bad = m >= 0x7F800000u;
  if (threadIdx.x == 0) scales[row] = rs.s;
  for (int col = threadIdx.x * 8; col < pitch; col += 8192)
    *reinterpret_cast<u32x2*>(codes + row * pitch + col) = bad ? u32x2{0u, 0u} : code8<DT>(load(col), rs.inv);
}

// fp32 rows to fp16 at a power of two each (w8a32_mm_t): 2^e takes a row's largest finite magnitude to
// [2^14, 2^15), so that none overflows and only what is 2^-39 of it or less becomes 0; back = -e.
// Columns cols .. pitch - 1 are 0.  One workgroup a row: a row is read twice, the second time from
// cache.  Bound by memory: 14 us of a call at [2048][4096], 51 at [1024][32000] (a cast 7 and 32).
__global__ __launch_bounds__(512) void half_rows_kernel(const float* __restrict__ X, int64_t cols, int64_t ld,
                                                        int64_t pitch, uint16_t* __restrict__ out,
                                                        int* __restrict__ back) {
  constexpr int T = 512;
  const int64_t row = blockIdx.x;
  const float* x = X + row * ld;
  auto load = [&](int64_t col) {
    if (col + 8 <= cols) return load_raw8<W4_DT_F32>(x + col);
    return col < cols ? load_raw8_part<W4_DT_F32>(x + col, (int)(cols - col), 0u) : Raw8<W4_DT_F32>{};
  };
  uint32_t m = 0;
#pragma unroll 4
  for (int64_t col = threadIdx.x * 8; col < cols; col += T * 8) {
    const Raw8<W4_DT_F32> r = load(col);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = r.q[j >> 2][j & 3] & 0x7FFFFFFFu;
      m = umax(m, u < 0x7F800000u ? u : 0u);
    }
  }
  m = wave_umax(m);
  __shared__ uint32_t part[T / 64];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < T / 64; ++i) m = umax(m, part[i]);
  const int e = m == 0 ? 0 : min(141 - (int)(m >> 23), 126);
  const float f = __uint_as_float((uint32_t)(127 + e) << 23);
  if (threadIdx.x == 0) back[row] = -e;
#pragma unroll 4
  for (int64_t col = threadIdx.x * 8; col < pitch; col += T * 8) {
    float v[8];
    widen8<W4_DT_F32>(load(col), v);
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack_f16x2(v[2 * j] * f, v[2 * j + 1] * f);
    *reinterpret_cast<u32x4*>(out + row * pitch + col) = o;
  }
}

template <int DT, int TPR, int C>
hipError_t launch(const void* X, int64_t rows, int cols, int64_t ld, int pitch, int8_t* codes, float* scales,
                  hipStream_t st) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  quantize_rows_kernel<DT, TPR, C><<<(unsigned)((rows + RPB - 1) / RPB), TPR < 256 ? 256 : TPR, 0, st>>>(
      X, rows, cols, ld, pitch, codes, scales);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const void* X, int64_t rows, int cols, int64_t ld, int pitch, int8_t* codes, float* scales,
                     hipStream_t st) {
  // chunks are counted over the pitch, so that the zero columns past `cols` are written too
  if (pitch <= 64 * 4 * 8) return launch<DT, 64, 4>(X, rows, cols, ld, pitch, codes, scales, st);
  if (pitch <= 256 * 4 * 8) return launch<DT, 256, 4>(X, rows, cols, ld, pitch, codes, scales, st);
  if (pitch <= 256 * 8 * 8) return launch<DT, 256, 8>(X, rows, cols, ld, pitch, codes, scales, st);
  quantize_long_rows_kernel<DT><<<(unsigned)rows, 1024, 0, st>>>(X, cols, ld, pitch, codes, scales);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_half_rows(const float* X, int64_t rows, int64_t cols, int64_t ld, uint16_t* out, int64_t pitch,
                            int* back, hipStream_t st) {
  // a launch holds fewer than 2^32 threads
  constexpr int64_t kRows = (int64_t)1 << 22;
  for (int64_t r = 0; r < rows; r += kRows) {
    half_rows_kernel<<<(unsigned)std::min(kRows, rows - r), 512, 0, st>>>(X + r * ld, cols, ld, pitch, out + r * pitch,
                                                                          back + r);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_quantize_rows(const void* X, int dt, int64_t rows, int64_t cols, int64_t ld, int8_t* codes,
                                float* scales, hipStream_t st) {
  const int pitch = (int)((cols + 63) / 64 * 64);
  // a launch holds fewer than 2^32 threads, a row takes at most 1024
  constexpr int64_t kRows = (int64_t)1 << 21;
  if (rows > kRows) {
    for (int64_t r = 0; r < rows; r += kRows) {
      const hipError_t e = launch_quantize_rows(static_cast<const char*>(X) + (size_t)(r * ld) * (dt == W4_DT_F32 ? 4 : 2), dt,
                                                std::min(kRows, rows - r), cols, ld, codes + (size_t)r * pitch, scales + r, st);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  switch (dt) {
    case W4_DT_F32: return launch_dt<W4_DT_F32>(X, rows, (int)cols, ld, pitch, codes, scales, st);
    case W4_DT_F16: return launch_dt<W4_DT_F16>(X, rows, (int)cols, ld, pitch, codes, scales, st);
    default: return launch_dt<W4_DT_BF16>(X, rows, (int)cols, ld, pitch, codes, scales, st);
  }
}

}  // namespace w4
