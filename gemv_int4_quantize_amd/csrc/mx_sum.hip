// Column sums of float rows (mx4_sum_rows: the bias's gradient of a linear layer), for gfx950:
//   out[n] = out_rne(sum_m X[m][n]), sums in fp32, in an order that M and N alone fix.
// Bound by reading X once.  A workgroup takes 256 columns and one of S runs of the rows: eight groups of
// 32 lanes, eight columns a lane, a row a group at a time (512 bytes of 16-bit elements next to one
// another).  Where the columns alone leave CUs idle the rows are shared, and the S sums are rows that a
// second launch sums: no atomics, and no counter that a captured graph would have to clear.
// 4096 x 11008 fp32 37.7 us (4.8 TB/s), 2048 x 4096 bf16 8.3 (two launches).
#include <algorithm>

#include "api_common.h"
#include "epilogue.h"
#include "launch.h"
#include "mx.h"

namespace w4 {

namespace {

constexpr int kCols = 256, kGroups = 8;

template <int DT>
__global__ __launch_bounds__(256) void mx_sum_kernel(const void* __restrict__ X, int64_t M, int N, int64_t ld, int64_t per,
                                                     const Epi ep, float* __restrict__ part) {
  typedef typename Elem<DT>::type E;
  __shared__ __attribute__((aligned(16))) float sums[kGroups][kCols];
  const int tid = threadIdx.x, group = tid >> 5, c = (blockIdx.x * (kCols / 8) + (tid & 31)) * 8;
  const int64_t m0 = blockIdx.y * per, m1 = std::min<int64_t>(M, m0 + per);
  float sum[8] = {};
  if (c < N) {
    const E* x = static_cast<const E*>(X);
#pragma unroll 4
    for (int64_t m = m0 + group; m < m1; m += kGroups) {
      float v[8];
      widen8<DT>(mx_chunk_of<DT>(x + m * ld, c, N), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[group][(tid & 31) * 8 + j] = sum[j];
  __syncthreads();
  const int n = blockIdx.x * kCols + tid;
  if (n >= N) return;
  float v = 0.0f;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) v += sums[g][tid];
  if (part != nullptr) part[(size_t)blockIdx.y * N + n] = v;
  else epi_put(ep, epi_col(ep, n), 0, v);
}

// Runs of the rows: two workgroups for each CU, of at least 64 rows.
int runs(int64_t M, int64_t N, const DeviceCaps& caps) {
  const int64_t blocks = (N + kCols - 1) / kCols;
  return (int)std::max<int64_t>(1, std::min<int64_t>(2 * caps.cus / blocks, M / 64));
}

template <int DT>
hipError_t run(const void* X, int64_t M, int64_t N, int64_t ld, int s, const Epi& ep, float* part, hipStream_t st) {
  mx_sum_kernel<DT><<<dim3((unsigned)((N + kCols - 1) / kCols), (unsigned)s), 256, 0, st>>>(X, M, (int)N, ld, (M + s - 1) / s, ep,
                                                                                           part);
  return hipGetLastError();
}

}  // namespace

size_t mx_sum_workspace_bytes(int64_t M, int64_t N, const DeviceCaps& caps) {
  const int s = runs(M, N, caps);
  return s > 1 ? (size_t)s * N * 4 : 0;
}

hipError_t launch_mx_sum(const void* X, int dt, int64_t M, int64_t N, int64_t ld, const Epi& ep, const DeviceCaps& caps, void* ws,
                         hipStream_t st) {
  const int s = runs(M, N, caps);
  float* part = s > 1 ? static_cast<float*>(ws) : nullptr;
  hipError_t e;
  switch (dt) {
    case W4_DT_F32: e = run<W4_DT_F32>(X, M, N, ld, s, ep, part, st); break;
    case W4_DT_F16: e = run<W4_DT_F16>(X, M, N, ld, s, ep, part, st); break;
    default: e = run<W4_DT_BF16>(X, M, N, ld, s, ep, part, st); break;
  }
  return e != hipSuccess || s == 1 ? e : run<W4_DT_F32>(part, s, N, N, 1, ep, nullptr, st);
}

}  // namespace w4
