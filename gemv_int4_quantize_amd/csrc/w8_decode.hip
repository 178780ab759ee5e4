// Product of int8 rows for one to four tokens (decode), for gfx950.  The weight is read once,
// from memory straight into matrix-core registers, and its bytes set the time; float tokens
// are quantized by the same launch.
//
// A workgroup of NW waves owns 16 channels; its waves share out the contraction in contiguous
// runs of 128-column units and add their sums through LDS.
// v_mfma_i32_16x16x64_i8 with channels as rows and tokens as columns: lane l supplies 16 bytes
// of channel l % 16 and of token l % 16, the same columns of both, and holds token l % 16 of
// channels 4 (l / 16) .. + 3.  Lane l takes the 32 bytes from column 32 (l / 16) of a unit for
// two products, so that each of its two loads touches whole 128-byte lines (half a line at a
// time, 64-column units, was slower).  The products cost 16 cycles for 1 KB of weight, so that
// most of the 16 token columns are idle does not matter.
// Measured, float tokens quantized in the launch: (N, K) = (12288, 4096), four tokens 15.8 us
// (3.2 TB/s: the start of a launch and the tokens' quantization take 4 us of it);
// (16384, 16384), two tokens 52 us, 5.1 TB/s; (2048, 2048), one token 5.5 us.
#include <algorithm>

#include "api_common.h"
#include "epilogue.h"
#include "launch.h"
#include "rows.h"

namespace w4 {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr int kNonTemporal = 2;  // cache-policy operand of a buffer load

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
template <int AUX>
__device__ __forceinline__ i32x4 load16(rsrc_t r, int off, int soff) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, AUX));
}

// Units of a lane's 32 columns (from column 32 q4 of each) that count.  The last unit of a pitch that
// is not a multiple of 128 holds 64 columns: past them the weight's bytes are the next channel's,
// and the tokens are taken as 0.
constexpr int code_cut(int pitch, int q4) {
  const int units = (pitch + 127) >> 7;
  return (pitch & 64) != 0 && q4 >= 2 ? units - 1 : units;
}
// Where a lane reads a token's codes for unit u: inside the token's row for every u, the last unit
// that counts standing in for those past it, and the first columns where none does (a pitch of 64).
constexpr int code_column(int cut, int q4) { return cut > 0 ? q4 * 32 : 0; }
constexpr int code_unit(int u, int cut) { return u < cut ? u : cut > 0 ? cut - 1 : 0; }
constexpr bool codes_in_row() {
  for (int pitch = 64; pitch <= 1024; pitch += 64)
    for (int q4 = 0; q4 < 4; ++q4)
      for (int u = 0; u < pitch / 128 + 9; ++u) {
        const int cut = code_cut(pitch, q4), at = code_column(cut, q4) + code_unit(u, cut) * 128;
        if (at < 0 || at + 32 > pitch) return false;
      }
  return true;
}
static_assert(codes_in_row(), "LDS reads of the token codes");

constexpr int kMaxM = 4;               // tokens
constexpr int kFusedLds = 64 * 1024;   // bytes of codes that a workgroup may hold

// XDT: -1: int8 tokens from memory; else the dtype of float tokens, quantized into LDS by every
// workgroup while its first weights are on their way.  Loads return in order, so the tokens
// are asked for before the weights: C chunks of eight of each token per thread (what is left
// of longer tokens is read twice).
// D units of a wave are in flight all the time: a unit's registers are loaded again as soon as
// its product is issued.  Past the wave's run the loads have an empty resource and give zeros
// without a request.
template <int NW, int D, int XDT, int C>
__global__ __launch_bounds__(NW * 64) void w8_decode_kernel(const int8_t* __restrict__ W, const float* __restrict__ sw,
                                                            const int8_t* __restrict__ A, const float* __restrict__ sa,
                                                            const void* __restrict__ X, int64_t ldx, int M, int N, int K,
                                                            int pitch, int first, const Epi ep) {
  constexpr int T = NW * 64;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ int sums[NW][kMaxM][16 + 4];
  __shared__ float tok_s[XDT >= 0 ? kMaxM : 1];
  __shared__ uint32_t part[XDT >= 0 ? kMaxM * NW : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = first + blockIdx.x * 16;
  const int units = (pitch + 127) >> 7;
  const int per = (units + NW - 1) / NW;
  const int u0 = min(wave * per, units), u1 = min(u0 + per, units);
  const int r16 = lane & 15, q4 = lane >> 4;

  const uint32_t wbytes = (uint32_t)min(16, N - n0) * (uint32_t)pitch;
  const int ow = r16 * pitch + q4 * 32;
  const int oa = min(r16, M - 1) * pitch + q4 * 32;
  i32x4 w[D][2], x[D][2];
  auto load = [&](int d, int u) {
    const bool in = u < u1;
    const rsrc_t rw = make_rsrc(W + (size_t)n0 * pitch, in ? wbytes : 0u);
#pragma unroll
    for (int h = 0; h < 2; ++h) w[d][h] = load16<kNonTemporal>(rw, ow + h * 16, u * 128);
    if constexpr (XDT < 0) {
      const rsrc_t ra = make_rsrc(A, in ? (uint32_t)M * (uint32_t)pitch : 0u);
#pragma unroll
      for (int h = 0; h < 2; ++h) x[d][h] = load16<0>(ra, oa + h * 16, u * 128);
    }
  };

  if constexpr (XDT >= 0) {
    typedef typename Elem<XDT>::type E;
    // token codes [M][pitch + 16]: the pad keeps the tokens' rows in distinct banks
    const int ch = pitch >> 3;
    auto chunk = [&](int m, int c) {
      const E* p = static_cast<const E*>(X) + m * ldx + c * 8;
      if (c * 8 + 8 <= K) return load_raw8<XDT>(p);
      return c * 8 < K ? load_raw8_part<XDT>(p, K - c * 8, 0u) : Raw8<XDT>{};
    };
    Raw8<XDT> held[kMaxM][C];
#pragma unroll
    for (int m = 0; m < kMaxM; ++m)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        held[m][c] = Raw8<XDT>{};
        if (m < M && tid + c * T < ch) held[m][c] = chunk(m, tid + c * T);
      }
    uint32_t am[kMaxM] = {};
#pragma unroll
    for (int m = 0; m < kMaxM; ++m)
      if (m < M)
        for (int c = tid + C * T; c < ch; c += T) am[m] = absmax8<XDT>(chunk(m, c), am[m]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, u0 + d);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < kMaxM; ++m) {
      if (m >= M) break;
#pragma unroll
      for (int c = 0; c < C; ++c) am[m] = absmax8<XDT>(held[m][c], am[m]);
      const uint32_t a = wave_umax(absmax_bits<XDT>(am[m]));
      if (lane == 0) part[m * NW + wave] = a;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kMaxM; ++m) {
      if (m >= M) break;
      uint32_t a = part[m * NW];
#pragma unroll
      for (int i = 1; i < NW; ++i) a = max(a, part[m * NW + i]);
      const RowScale rs = row_scale(a);
      const bool bad = a >= 0x7F800000u;
      if (tid == 0) tok_s[m] = rs.s;
      auto put = [&](int c, const Raw8<XDT>& r) {
        *reinterpret_cast<u32x2*>(smem + m * (pitch + 16) + c * 8) = bad ? u32x2{0u, 0u} : code8<XDT>(r, rs.inv);
      };
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (tid + c * T < ch) put(tid + c * T, held[m][c]);
      for (int c = tid + C * T; c < ch; c += T) put(c, chunk(m, c));
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, u0 + d);
  }

  i32x4 acc = {0, 0, 0, 0};
  const int cut = code_cut(pitch, q4);
  const char* xl = smem + min(r16, M - 1) * (pitch + 16) + code_column(cut, q4);
  for (int u = u0; u < u1; u += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (XDT >= 0) {
          // past the wave's run the weight is 0
          x[d][h] = *reinterpret_cast<const i32x4*>(xl + code_unit(u + d, cut) * 128 + h * 16);
        }
        const i32x4 t = u + d < cut ? x[d][h] : i32x4{0, 0, 0, 0};
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[d][h], t, acc, 0, 0, 0);
      }
      load(d, u + D + d);
    }
  }
  if (r16 < M) *reinterpret_cast<i32x4*>(&sums[wave][r16][q4 * 4]) = acc;
  __syncthreads();
  const int m = tid >> 4, n = tid & 15;
  if (m >= M || n0 + n >= N) return;
  int s = 0;
#pragma unroll
  for (int v = 0; v < NW; ++v) s += sums[v][m][n];
  epi_put(ep, epi_col(ep, n0 + n), m, w8_scaled(s, XDT >= 0 ? tok_s[m] : sa[m], sw[n0 + n]));
}

template <int NW, int D, int XDT, int C>
hipError_t run(const W8Args& a, hipStream_t st) {
  const size_t lds = XDT >= 0 ? (size_t)a.M * (a.pitch + 16) : 0;
  auto k = w8_decode_kernel<NW, D, XDT, C>;
  if (lds > 48 * 1024) {  // with the static part over 64 KB
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  // a launch holds fewer than 2^32 threads
  constexpr int64_t kChannels = (int64_t)1 << 25;
  for (int64_t n = 0; n < a.N; n += kChannels) {
    const int64_t wgs = (std::min(kChannels, a.N - n) + 15) / 16;
    k<<<(unsigned)wgs, NW * 64, lds, st>>>(a.W, a.w_scales, a.A, a.a_scales, a.X, a.ldx, (int)a.M, (int)a.N, (int)a.K,
                                           (int)a.pitch, (int)n, a.ep);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Sixteen waves a workgroup where there are few workgroups (less than two a CU), else eight.
template <int XDT>
hipError_t run_x(const W8Args& a, const DeviceCaps& caps, hipStream_t st) {
  const bool few = a.N < 16 * 2 * (int64_t)caps.cus;
  if (XDT < 0) return few ? run<16, 4, XDT, 1>(a, st) : run<8, 4, XDT, 1>(a, st);
  if (few) return a.pitch <= 8192 ? run<16, 4, XDT, 1>(a, st) : run<16, 4, XDT, 2>(a, st);
  return a.pitch <= 4096 ? run<8, 4, XDT, 1>(a, st) : run<8, 4, XDT, 3>(a, st);
}

}  // namespace

bool w8_fused(int64_t M, int64_t K) {
  return M <= kMaxM && M * ((K + 63) / 64 * 64 + 16) <= kFusedLds;
}

// More tokens than these run on the tiles: at 16 tokens the 64 x 64 tile takes 16 us on
// (N, K) = (12288, 4096), this kernel's form for 16 took 19.5.
bool w8_decode_supported(int64_t M) { return M <= kMaxM; }

hipError_t launch_w8_decode(const W8Args& a, const DeviceCaps& caps, hipStream_t st) {
  if (a.X == nullptr) return run_x<-1>(a, caps, st);
  switch (a.x_dt) {
    case W4_DT_F32: return run_x<W4_DT_F32>(a, caps, st);
    case W4_DT_F16: return run_x<W4_DT_F16>(a, caps, st);
    default: return run_x<W4_DT_BF16>(a, caps, st);
  }
}

}  // namespace w4
