// Product of int8 rows with a scale for each token and channel, for gfx950:
//   Y[m][n] = out_rne((fp32(sum_k A[m][k] W[n][k]) * w_scales[n]) * a_scales[m] + bias[n]),
// the sum exact in int32 (K < 2^17 keeps 128 * 128 * K below 2^31).
#include <cstdlib>

#include "api_common.h"
#include "epilogue.h"
#include "launch.h"
#include "rows.h"

namespace w4 {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void;

// raw buffer resource (gfx9-class dword 3: 32-bit data format); loads past `bytes` read 0
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

constexpr int kBK = 64;  // contraction columns (bytes) of a stage

// One workgroup of WM x WN waves computes a (WM FM 32) x (WN FN 32) tile.  Both operands run
// along the contraction, so a stage (64 columns of every row of both tiles) goes global -> LDS
// with direct loads, through a ring of NB stages: NB - 2 stages are in flight while one is
// computed.  A stage's rows are 64 bytes, their 16-byte chunk index XOR-ed with (row / 2) % 4,
// so that eight lanes' operand reads fall in distinct banks; the XOR is on the source address, since a
// direct load writes 64 consecutive chunks.
// v_mfma_i32_32x32x32_i8: lane l supplies 16 bytes of row l % 32 of each operand (columns
// 16 (l / 32) ..), and holds column l % 32 of the result, register r being row 8 (r / 4) +
// 4 (l / 32) + (r % 4).  The operands of a half stage are read during the products of the
// half before it, across the barrier too, and one barrier a stage is enough: behind it every
// wave has read the stage that the next direct load overwrites.
template <int WM, int WN, int FM, int FN, int NB>
__global__ __launch_bounds__(WM * WN * 64) void w8_ring_kernel(const int8_t* __restrict__ A, const float* __restrict__ sa,
                                                               const int8_t* __restrict__ W, const float* __restrict__ sw,
                                                               const Epi ep, int M, int N, int pitch, int tm, int tn) {
  constexpr int T = WM * WN * 64, BM = WM * FM * 32, BN = WN * FN * 32;
  constexpr int UA = BM * 4 / T, UB = BN * 4 / T;  // chunks a thread loads of each tile in a stage
  constexpr int STAGE = (BM + BN) * kBK;
  static_assert(BM * 4 % T == 0 && BN * 4 % T == 0, "tile split");
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int m0 = (blockIdx.x % tm) * BM, n0 = (blockIdx.x / tm) * BN;

  const rsrc_t ra = make_rsrc(A + (size_t)m0 * pitch, (uint32_t)min(BM, M - m0) * (uint32_t)pitch);
  const rsrc_t rb = make_rsrc(W + (size_t)n0 * pitch, (uint32_t)min(BN, N - n0) * (uint32_t)pitch);
  int oa[UA], ob[UB];
#pragma unroll
  for (int i = 0; i < UA; ++i) {
    const int u = tid + i * T, row = u >> 2;
    oa[i] = row * pitch + (((u & 3) ^ ((row >> 1) & 3)) << 4);
  }
#pragma unroll
  for (int i = 0; i < UB; ++i) {
    const int u = tid + i * T, row = u >> 2;
    ob[i] = row * pitch + (((u & 3) ^ ((row >> 1) & 3)) << 4);
  }
  const int KT = pitch / kBK;
  // stage kt into ring slot `slot`; past the end it loads the last stage, which is never read
  // (the casts to int: without them the host pass drops the launch stub)
  auto dma = [&](int kt, int slot) {
    const int so = min(kt, KT - 1) * kBK;
    char* base = smem + slot * STAGE + wave * 1024;
#pragma unroll
    for (int i = 0; i < UA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(base + i * T * 16), 16, (int)oa[i], (int)so, 0, 0);
#pragma unroll
    for (int i = 0; i < UB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(base + BM * kBK + i * T * 16), 16, (int)ob[i], (int)so, 0, 0);
  };
  // all but the last NB - 2 stages landed and this wave's reads done, then a barrier with no
  // fence (a fence would wait for every load in flight)
  auto sync = [&]() {
    constexpr int n = (NB - 2) * (UA + UB);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((n & 15) | 0x70 | ((n >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  const int lr = lane & 31, hi = lane >> 5, sx = (lr >> 1) & 3;
  // the fragment's byte offset in its tile for the first half stage; the second half is ^ 32
  const int fa = (wm * FM * 32 + lr) * kBK + ((hi ^ sx) << 4);
  const int fb = BM * kBK + (wn * FN * 32 + lr) * kBK + ((hi ^ sx) << 4);
  auto read = [&](int slot, int kk, u32x4 (&x)[FM], u32x4 (&y)[FN]) {
    const char* base = smem + slot * STAGE;
#pragma unroll
    for (int i = 0; i < FM; ++i) x[i] = *reinterpret_cast<const u32x4*>(base + (fa ^ (kk * 32)) + i * 32 * kBK);
#pragma unroll
    for (int j = 0; j < FN; ++j) y[j] = *reinterpret_cast<const u32x4*>(base + (fb ^ (kk * 32)) + j * 32 * kBK);
  };
  i32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  auto mul = [&](const u32x4 (&x)[FM], const u32x4 (&y)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, x[i]), __builtin_bit_cast(i32x4, y[j]),
                                                          acc[i][j], 0, 0, 0);
  };
  u32x4 x0[FM], y0[FN], x1[FM], y1[FN];
#pragma unroll
  for (int k = 0; k < NB - 1; ++k) dma(k, k);
  sync();
  dma(NB - 1, NB - 1);
  read(0, 0, x0, y0);
  read(0, 1, x1, y1);
  mul(x0, y0);
  int slot = 1;
  for (int kt = 1; kt < KT; ++kt) {
    sync();
    dma(kt + NB - 1, slot == 0 ? NB - 1 : slot - 1);
    // the order of issue as written: left to itself the compiler delays the reads until the
    // products before them have freed their registers
    read(slot, 0, x0, y0);
    __builtin_amdgcn_sched_barrier(0);
    mul(x1, y1);
    __builtin_amdgcn_sched_barrier(0);
    read(slot, 1, x1, y1);
    __builtin_amdgcn_sched_barrier(0);
    mul(x0, y0);
    slot = slot == NB - 1 ? 0 : slot + 1;
  }
  mul(x1, y1);
  // no direct LDS load may land after the workgroup's LDS is handed on
  __builtin_amdgcn_s_waitcnt(0x0070);

  const int rbase = m0 + wm * FM * 32 + hi * 4;
  const int cbase = n0 + wn * FN * 32;
  const bool wide = epi_wide(ep, N) != 0;
  const rsrc_t rs = make_rsrc(sa, (uint32_t)M * 4u);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    float s[16];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (rbase + i * 32 + g * 8) * 4, 0, 0));
#pragma unroll
      for (int q = 0; q < 4; ++q) s[g * 4 + q] = __uint_as_float(v[q]);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int c = cbase + j * 32 + lr;
      const float w = c < N ? sw[c] : 0.0f;
      f32x16 o;
#pragma unroll
      for (int r = 0; r < 16; ++r) o[r] = w8_scaled(acc[i][j][r], s[r], w);
      if (wide) {
        epi_put_block_wide(epi_quad(ep, cbase + j * 32 + (lr & ~3), N), o, rbase + i * 32, M, lane);
      } else if (c < N) {
        const EpiCol col = epi_col(ep, c);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int m = rbase + i * 32 + (r >> 2) * 8 + (r & 3);
          if (m < M) epi_put(ep, col, m, o[r]);
        }
      }
    }
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

namespace {

template <int WM, int WN, int FM, int FN, int NB>
hipError_t run_ring(const W8Args& a, hipStream_t st) {
  constexpr int BM = WM * FM * 32, BN = WN * FN * 32;
  auto k = w8_ring_kernel<WM, WN, FM, FN, NB>;
  constexpr int lds = NB * (BM + BN) * kBK;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int64_t tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
  k<<<(unsigned)(tm * tn), WM * WN * 64, lds, st>>>(a.A, a.a_scales, a.W, a.w_scales, a.ep, (int)a.M, (int)a.N,
                                                    (int)a.pitch, (int)tm, (int)tn);
  return hipGetLastError();
}

}  // namespace

size_t w8_mm_workspace_bytes(int64_t, int64_t, int64_t, const DeviceCaps&) { return 0; }

const char* w8_mm_name(int64_t, int64_t, int64_t, const DeviceCaps&) { return "w8_ring"; }

hipError_t launch_w8_mm(const W8Args& a, const DeviceCaps&, void*, size_t, hipStream_t st) {
  static const char* e = getenv("W8A8_CFG");
  const int cfg = e ? atoi(e) : (a.M > 256 ? 0 : 3);
  switch (cfg) {
    case 0: return run_ring<2, 4, 4, 2, 4>(a, st);
    case 1: return run_ring<2, 2, 4, 4, 4>(a, st);
    case 2: return run_ring<2, 2, 4, 2, 3>(a, st);
    case 3: return run_ring<2, 2, 2, 2, 4>(a, st);
    case 4: return run_ring<2, 2, 1, 1, 4>(a, st);
    case 5: return run_ring<2, 2, 4, 2, 4>(a, st);
    case 6: return run_ring<2, 4, 4, 2, 5>(a, st);
    default: return run_ring<2, 4, 2, 2, 4>(a, st);
  }
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
