// Product of int8 rows with a scale for each token and channel, for gfx950:
//   Y[m][n] = out_rne((fp32(sum_k A[m][k] W[n][k]) * w_scales[n]) * a_scales[m] + bias[n]),
// the sum exact in int32 (K < 2^17 keeps 128 * 128 * K below 2^31).
#include "api_common.h"
#include "epilogue.h"
#include "launch.h"
#include "rows.h"

namespace w4 {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// One workgroup of four waves (2 x 2) computes a 64 x 64 tile, staged through LDS 64 columns
// at a time.  v_mfma_i32_32x32x32_i8: lane l supplies 16 bytes of row l % 32 of each operand
// (columns 16 (l / 32) ..), and holds column l % 32 of the result, register r being row
// 8 (r / 4) + 4 (l / 32) + (r % 4).
__global__ __launch_bounds__(256) void w8_tile_kernel(const int8_t* __restrict__ A, const float* __restrict__ sa,
                                                      const int8_t* __restrict__ W, const float* __restrict__ sw,
                                                      const Epi ep, int M, int N, int pitch) {
  __shared__ u32x4 As[64 * 5], Bs[64 * 5];  // rows of 64 bytes, padded to 80
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int row = tid >> 2, ch = tid & 3;
  const u32x4* ga = reinterpret_cast<const u32x4*>(A + (size_t)min(m0 + row, M - 1) * pitch) + ch;
  const u32x4* gb = reinterpret_cast<const u32x4*>(W + (size_t)min(n0 + row, N - 1) * pitch) + ch;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  i32x16 acc = {};
  for (int k = 0; k < pitch; k += 64) {
    const u32x4 a = ga[k >> 4], b = gb[k >> 4];
    __syncthreads();
    As[row * 5 + ch] = a;
    Bs[row * 5 + ch] = b;
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const u32x4 x = As[(wm + (lane & 31)) * 5 + kk * 2 + (lane >> 5)];
      const u32x4 y = Bs[(wn + (lane & 31)) * 5 + kk * 2 + (lane >> 5)];
      acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, x), __builtin_bit_cast(i32x4, y), acc, 0, 0, 0);
    }
  }
  const int n = n0 + wn + (lane & 31);
  if (n >= N) return;
  const EpiCol col = epi_col(ep, n);
  const float s = sw[n];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int m = m0 + wm + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
    if (m < M) epi_put(ep, col, m, w8_scaled(acc[r], sa[m], s));
  }
}

// dY rows copied to an aligned pitch, zeros past column N (w8a16_mm_t).
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ x, int64_t N, int64_t ld,
                                                       uint16_t* __restrict__ out, int64_t npad) {
  const int64_t row = blockIdx.y;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= npad) return;
  const uint16_t* p = x + row * ld + c;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (c + 8 <= N) v = load_raw8<W4_DT_BF16>(p).q[0];
  else if (c < N) v = load_raw8_part<W4_DT_BF16>(p, (int)(N - c), 0u).q[0];
  *reinterpret_cast<u32x4*>(out + row * npad + c) = v;
}

}  // namespace

size_t w8_mm_workspace_bytes(int64_t, int64_t, int64_t, const DeviceCaps&) { return 0; }

const char* w8_mm_name(int64_t, int64_t, int64_t, const DeviceCaps&) { return "w8_64x64"; }

hipError_t launch_w8_mm(const W8Args& a, const DeviceCaps&, void*, size_t, hipStream_t st) {
  const dim3 grid((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 63) / 64));
  w8_tile_kernel<<<grid, 256, 0, st>>>(a.A, a.a_scales, a.W, a.w_scales, a.ep, (int)a.M, (int)a.N, (int)a.pitch);
  return hipGetLastError();
}

hipError_t launch_pad_rows(const uint16_t* dY, int64_t M, int64_t N, int64_t ld, uint16_t* out, int64_t npad,
                           hipStream_t st) {
  // grid.y is limited to 65535 rows a launch
  for (int64_t m = 0; m < M; m += 32768) {
    const int64_t n = M - m < 32768 ? M - m : 32768;
    pad_rows_kernel<<<dim3((unsigned)((npad / 8 + 255) / 256), (unsigned)n), 256, 0, st>>>(dY + m * ld, N, ld,
                                                                                           out + m * npad, npad);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace w4
