// Product of microscaled 4-bit rows for a few tokens (decode), for gfx950.  The weight is read once,
// from memory straight into matrix-core registers, and its bytes set the time; up to four float
// tokens are quantized by the same launch.
//
// A workgroup of NW waves owns 16 channels; its waves share out the contraction in contiguous runs
// of 256-column units and add their sums through LDS.
// v_mfma_scale_f32_16x16x128_f8f6f4 with channels as rows and tokens as columns: lane l supplies a
// block of 32 columns of channel l % 16 and of token l % 16, the same columns of both, and their two
// exponents, and holds token l % 16 of channels 4 (l / 16) .. + 3.  Lane l takes the two blocks
// from column 64 (l / 16) of a unit for two products, so that its loads touch whole 128-byte lines.
#include <algorithm>

#include "api_common.h"
#include "epilogue.h"
#include "launch.h"
#include "mx.h"

namespace w4 {

namespace {

constexpr int kNonTemporal = 2;  // cache-policy operand of a buffer load

template <int AUX>
__device__ __forceinline__ u32x4 load16(rsrc_t r, int off, int soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, AUX));
}

constexpr int kMaxM = 16;             // tokens
constexpr int kMaxFused = 4;          // of them quantized by the launch
constexpr int kFusedLds = 64 * 1024;  // bytes of codes and exponents that a workgroup may hold

// Units of a lane's 64 columns (from column 64 q4 of each) that count.  The last unit of a row of
// P columns that is not a multiple of 256 holds 128: past them the weight's bytes are the next
// channel's, and both operands are taken as 0.
constexpr int live_units(int P, int q4) {
  const int units = (P + 255) >> 8;
  return (P & 128) != 0 && q4 >= 2 ? units - 1 : units;
}
// Where a lane reads a token's row for unit u (in 64-column pieces): inside the row for every u.
constexpr int token_piece(int u, int live, int q4) { return live <= 0 ? 0 : (u < live ? u : live - 1) * 4 + q4; }
constexpr bool pieces_in_row() {
  for (int P = 128; P <= 2048; P += 128)
    for (int q4 = 0; q4 < 4; ++q4)
      for (int u = 0; u < P / 256 + 9; ++u) {
        const int at = token_piece(u, live_units(P, q4), q4);
        if (at < 0 || (at + 1) * 64 > P) return false;
      }
  return true;
}
static_assert(pieces_in_row(), "LDS reads of the tokens' codes");

// XDT: -1: tokens' codes from memory; else the dtype of float tokens, quantized into LDS by every
// workgroup while its first weights are on their way.  Loads return in order, so the tokens are
// asked for before the weights: C chunks of eight of each token per thread (what is left of longer
// tokens is read behind them).
// D units of a wave are in flight all the time: a unit's registers are loaded again as soon as its
// products are issued.  Past the wave's run the loads have an empty resource and give zeros
// without a request.
template <int NW, int D, int XDT, int C>
__global__ __launch_bounds__(NW * 64) void mx_decode_kernel(const uint8_t* __restrict__ W, const uint8_t* __restrict__ we,
                                                            const uint8_t* __restrict__ A, const uint8_t* __restrict__ ae,
                                                            const void* __restrict__ X, int64_t ldx, int M, int N, int K,
                                                            int P, int first, const Epi ep) {
  constexpr int T = NW * 64;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ float sums[NW][XDT >= 0 ? kMaxFused : kMaxM][16 + 4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = first + blockIdx.x * 16;
  const int units = (P + 255) >> 8;
  const int per = (units + NW - 1) / NW;
  const int u0 = min(wave * per, units), u1 = min(u0 + per, units);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int row = P >> 1, erow = P >> 5;  // bytes of a row's codes and exponents

  const uint32_t channels = (uint32_t)min(16, N - n0);
  const int ow = r16 * row + q4 * 32, oe = r16 * erow + q4 * 2;
  const int m0 = min(r16, M - 1);
  u32x4 w[D][2], x[D][2];
  uint32_t se[D], sx[D];
  auto load = [&](int d, int u) {
    const bool in = u < u1;
    const rsrc_t rw = mx_rsrc(W + (size_t)n0 * row, in ? channels * (uint32_t)row : 0u);
    const rsrc_t re = mx_rsrc(we + (size_t)n0 * erow, in ? channels * (uint32_t)erow : 0u);
#pragma unroll
    for (int h = 0; h < 2; ++h) w[d][h] = load16<kNonTemporal>(rw, ow + h * 16, u * 128);
    se[d] = __builtin_amdgcn_raw_buffer_load_b16(re, oe, u * 8, 0);
    if constexpr (XDT < 0) {
      const rsrc_t ra = mx_rsrc(A, in ? (uint32_t)M * (uint32_t)row : 0u);
      const rsrc_t rx = mx_rsrc(ae, in ? (uint32_t)M * (uint32_t)erow : 0u);
#pragma unroll
      for (int h = 0; h < 2; ++h) x[d][h] = load16<0>(ra, m0 * row + q4 * 32 + h * 16, u * 128);
      sx[d] = __builtin_amdgcn_raw_buffer_load_b16(rx, m0 * erow + q4 * 2, u * 8, 0);
    }
  };

  // in LDS: exponents [M][erow], then codes [M][row + 16] (the pad keeps the tokens' rows in distinct banks)
  const int codes_at = (M * erow + 15) & ~15;
  if constexpr (XDT >= 0) {
    typedef typename Elem<XDT>::type E;
    const int ch = P >> 3;
    auto chunk = [&](int m, int c) {
      const E* p = static_cast<const E*>(X) + m * ldx + c * 8;
      if (c * 8 + 8 <= K) return load_raw8<XDT>(p);
      return c * 8 < K ? load_raw8_part<XDT>(p, K - c * 8, 0u) : Raw8<XDT>{};
    };
    auto put = [&](int m, int c, const Raw8<XDT>& r) {
      uint32_t e;
      const uint32_t code = mx_chunk<XDT>(r, &e);
      if (c < ch) {
        *reinterpret_cast<uint32_t*>(smem + codes_at + m * (row + 16) + c * 4) = code;
        if ((c & 3) == 0) smem[m * erow + (c >> 2)] = (char)e;
      }
    };
    Raw8<XDT> held[kMaxFused][C];
#pragma unroll
    for (int m = 0; m < kMaxFused; ++m)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        held[m][c] = Raw8<XDT>{};
        if (m < M && tid + c * T < ch) held[m][c] = chunk(m, tid + c * T);
      }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, u0 + d);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < kMaxFused; ++m) {
      if (m >= M) break;
#pragma unroll
      for (int c = 0; c < C; ++c) put(m, tid + c * T, held[m][c]);
      for (int c = tid + C * T; c - tid < ch; c += T) put(m, c, c < ch ? chunk(m, c) : Raw8<XDT>{});
    }
    // this wave's LDS writes done, then a barrier with no fence, which would wait for the weights
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  } else {
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, u0 + d);
  }

  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  const int live = live_units(P, q4);
  const char* xc = smem + codes_at + m0 * (row + 16);
  const char* xe = smem + m0 * erow;
  for (int u = u0; u < u1; u += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if constexpr (XDT >= 0) {
        const int at = token_piece(u + d, live, q4);  // past the wave's run the weight is 0
#pragma unroll
        for (int h = 0; h < 2; ++h) x[d][h] = *reinterpret_cast<const u32x4*>(xc + at * 32 + h * 16);
        sx[d] = *reinterpret_cast<const uint16_t*>(xe + at * 2);
      }
      const bool in = u + d < live;
      const int ew = in ? (int)se[d] : 0, ex = in ? (int)sx[d] : 0;
      const u32x4 z = {0u, 0u, 0u, 0u};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(in ? w[d][0] : z), mx_operand(x[d][0]), acc, kFp4, kFp4,
                                                             0, ew, 0, ex);
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(in ? w[d][1] : z), mx_operand(x[d][1]), acc, kFp4, kFp4,
                                                             1, ew, 1, ex);
      load(d, u + D + d);
    }
  }
  if (r16 < M) *reinterpret_cast<f32x4*>(&sums[wave][r16][q4 * 4]) = acc;
  __syncthreads();
  const int m = tid >> 4, n = tid & 15;
  if (m >= M || n0 + n >= N) return;
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < NW; ++v) s += sums[v][m][n];
  epi_put(ep, epi_col(ep, n0 + n), m, s);
}

size_t fused_lds(int64_t M, int64_t P) { return ((M * (P >> 5) + 15) & ~15) + M * ((P >> 1) + 16); }

template <int NW, int D, int XDT, int C>
hipError_t run(const MxArgs& a, hipStream_t st) {
  const size_t lds = XDT >= 0 ? fused_lds(a.M, a.P) : 0;
  auto k = mx_decode_kernel<NW, D, XDT, C>;
  if (lds > 48 * 1024) {  // with the static part over 64 KB
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  // a launch holds fewer than 2^32 threads
  constexpr int64_t kChannels = (int64_t)1 << 25;
  for (int64_t n = 0; n < a.N; n += kChannels) {
    const int64_t wgs = (std::min(kChannels, a.N - n) + 15) / 16;
    k<<<(unsigned)wgs, NW * 64, lds, st>>>(a.W, a.w_scales, a.A, a.a_scales, a.X, a.ldx, (int)a.M, (int)a.N, (int)a.K,
                                           (int)a.P, (int)n, a.ep);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Sixteen waves a workgroup where there are few workgroups (less than two a CU), else eight.
template <int XDT>
hipError_t run_x(const MxArgs& a, const DeviceCaps& caps, hipStream_t st) {
  const bool few = a.N < 16 * 2 * (int64_t)caps.cus;
  if (XDT < 0) return few ? run<16, 4, XDT, 1>(a, st) : run<8, 4, XDT, 1>(a, st);
  if (few) return a.P <= 8192 ? run<16, 4, XDT, 1>(a, st) : run<16, 4, XDT, 2>(a, st);
  return a.P <= 4096 ? run<8, 4, XDT, 1>(a, st) : run<8, 4, XDT, 3>(a, st);
}

}  // namespace

bool mx_fused(int64_t M, int64_t K) { return M <= kMaxFused && fused_lds(M, mx_pitch(K)) <= (size_t)kFusedLds; }

bool mx_decode_supported(int64_t M) { return M <= kMaxM; }

hipError_t launch_mx_decode(const MxArgs& a, const DeviceCaps& caps, hipStream_t st) {
  if (a.X == nullptr) return run_x<-1>(a, caps, st);
  switch (a.x_dt) {
    case W4_DT_F32: return run_x<W4_DT_F32>(a, caps, st);
    case W4_DT_F16: return run_x<W4_DT_F16>(a, caps, st);
    default: return run_x<W4_DT_BF16>(a, caps, st);
  }
}

}  // namespace w4
