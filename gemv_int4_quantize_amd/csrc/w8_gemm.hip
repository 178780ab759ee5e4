// Product of int8 rows with a scale for each token and channel, for gfx950:
//   Y[m][n] = out_rne((fp32(sum_k A[m][k] W[n][k]) * w_scales[n]) * a_scales[m] + bias[n]),
// the sum exact in int32 (K < 2^17 keeps 128 * 128 * K below 2^31).
#include <algorithm>
#include <cstdio>

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

// Contraction columns (bytes) of a stage: two 64-byte halves of a row asked for one after the
// other cost more than the 128-byte line at once (measured at M = 2048, (N, K) = (4096, 11008)
// with 256 x 128 tiles: 116 us with 64-column stages, 99 us with these).
constexpr int BK = 128;

// One workgroup of WM x WN waves computes a (WM FM 32) x (WN FN 32) tile.  Both operands run
// along the contraction, so a stage (BK columns of every row of both tiles) goes global -> LDS
// with direct loads, through a ring of NB stages.  A stage's rows are 128 bytes, their 16-byte
// chunk index XOR-ed with (row / 2) % 8: a 16-byte LDS read takes lanes 0-3, 12-15 and 20-27
// (and so on, sixteen at a time) over 64 banks at once, and these then hit distinct ones (no
// bank conflict counted).  The XOR is on the source address, since a direct load writes 64
// consecutive chunks.
// v_mfma_i32_32x32x32_i8: lane l supplies 16 bytes of row l % 32 of each operand (columns
// 16 (l / 32) ..), and holds column l % 32 of the result, register r being row 8 (r / 4) +
// 4 (l / 32) + (r % 4).
// The one barrier a stage says that the stage has landed for every wave, and that every wave
// has read the stage before it, whose slot the direct loads of this stage then fill.  The
// stage's first operands are read behind the barrier while the last products of the stage
// before it run.
// What bounds it: at 8192^3 2359 TOP/s; the matrix cores are busy 68% of the cycles and the
// clock is down to 1.65 GHz under the load (the same product of zeros runs 1.2 times faster).
template <int WM, int WN, int FM, int FN, int NB>
__device__ __forceinline__ void ring_tile(char* smem, const int8_t* __restrict__ A, const float* __restrict__ sa,
                                          const int8_t* __restrict__ W, const float* __restrict__ sw, const Epi& ep, int M,
                                          int N, int pitch, int m0, int n0, int slice, int kt_per_slice,
                                          int* __restrict__ part) {
  constexpr int T = WM * WN * 64, BM = WM * FM * 32, BN = WN * FN * 32;
  constexpr int CH = BK / 16, UA = BM * CH / T, UB = BN * CH / T;  // chunks a thread loads of each tile in a stage
  constexpr int STAGE = (BM + BN) * BK;
  constexpr int SUB = BK / 32;  // products along a stage
  auto swz = [](int row) { return (row >> 1) & 7; };
  static_assert(BM * CH % T == 0 && BN * CH % T == 0, "tile split");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const rsrc_t ra = make_rsrc(A + (size_t)m0 * pitch, (uint32_t)min(BM, M - m0) * (uint32_t)pitch);
  const rsrc_t rb = make_rsrc(W + (size_t)n0 * pitch, (uint32_t)min(BN, N - n0) * (uint32_t)pitch);
  int oa[UA], ob[UB];
#pragma unroll
  for (int i = 0; i < UA; ++i) {
    const int u = tid + i * T, row = u / CH;
    oa[i] = row * pitch + (((u % CH) ^ swz(row)) << 4);
  }
#pragma unroll
  for (int i = 0; i < UB; ++i) {
    const int u = tid + i * T, row = u / CH;
    ob[i] = row * pitch + (((u % CH) ^ swz(row)) << 4);
  }
  // this slice's stages
  const int k0 = slice * kt_per_slice;
  const int KT = min((pitch + BK - 1) / BK - k0, kt_per_slice);
  // stage kt into ring slot `slot`; past the end it loads the last stage, which is never read
  // (the casts to int: without them the host pass drops the launch stub)
  auto dma_part = [&](int kt, int slot, int lo, int hi) {
    const int so = (k0 + min(kt, KT - 1)) * BK;
    char* base = smem + slot * STAGE + wave * 1024;
#pragma unroll
    for (int i = 0; i < UA + UB; ++i) {
      if (i < lo || i >= hi) continue;
      if (i < UA)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(base + i * T * 16), 16, (int)oa[i < UA ? i : 0], (int)so, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(base + BM * BK + (i - UA) * T * 16), 16,
                                                 (int)ob[i < UA ? 0 : i - UA], (int)so, 0, 0);
    }
  };
  auto dma = [&](int kt, int slot) { dma_part(kt, slot, 0, UA + UB); };
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
  const int lr = lane & 31, hi = lane >> 5, sx = swz(lr);
  // the fragment's byte offset in its tile at the start of a stage; product p is at ^ 32 p
  const int fa = (wm * FM * 32 + lr) * BK + ((hi ^ sx) << 4);
  const int fb = BM * BK + (wn * FN * 32 + lr) * BK + ((hi ^ sx) << 4);
  auto read = [&](int slot, int kk, u32x4 (&x)[FM], u32x4 (&y)[FN]) {
    const char* base = smem + slot * STAGE;
#pragma unroll
    for (int i = 0; i < FM; ++i) x[i] = *reinterpret_cast<const u32x4*>(base + (fa ^ (kk * 32)) + i * 32 * BK);
#pragma unroll
    for (int j = 0; j < FN; ++j) y[j] = *reinterpret_cast<const u32x4*>(base + (fb ^ (kk * 32)) + j * 32 * BK);
  };
  i32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  auto mul1 = [](const u32x4& x, const u32x4& y, i32x16& c) {
    c = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, x), __builtin_bit_cast(i32x4, y), c, 0, 0, 0);
  };
  auto mul = [&](const u32x4 (&x)[FM], const u32x4 (&y)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) mul1(x[i], y[j], acc[i][j]);
  };
  // Registers of even and odd products alternate: one set is multiplied while the other is
  // read.  The order of issue is as written: left to itself the compiler delays the reads
  // until the products before them have freed their registers, and bunches the direct loads,
  // and the matrix cores wait for both.
  u32x4 x[2][FM], y[2][FN];
#pragma unroll
  for (int k = 0; k < NB - 1; ++k) dma(k, k);
  int slot = 0;
  for (int kt = 0; kt < KT; ++kt) {
    sync();
    read(slot, 0, x[0], y[0]);
    __builtin_amdgcn_sched_barrier(0);
    const int free_slot = slot == 0 ? NB - 1 : slot - 1;
    const char* base = smem + slot * STAGE;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      // the last products of the stage before, their registers refilled one by one
      if (kt > 0) {
#pragma unroll
        for (int j = 0; j < FN; ++j) mul1(x[1][i], y[1][j], acc[i][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
      dma_part(kt + NB - 1, free_slot, i * (UA + UB) / FM, (i + 1) * (UA + UB) / FM);
      x[1][i] = *reinterpret_cast<const u32x4*>(base + (fa ^ 32) + i * 32 * BK);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) y[1][j] = *reinterpret_cast<const u32x4*>(base + (fb ^ 32) + j * 32 * BK);
    __builtin_amdgcn_sched_barrier(0);
    mul(x[0], y[0]);
    if ((k0 + kt) * BK + 64 < pitch)  // the row's last stage may be half a one
#pragma unroll
    for (int p = 2; p < SUB; ++p) {
      __builtin_amdgcn_sched_barrier(0);
      read(slot, p, x[p & 1], y[p & 1]);
      __builtin_amdgcn_sched_barrier(0);
      mul(x[(p - 1) & 1], y[(p - 1) & 1]);
    }
    slot = slot == NB - 1 ? 0 : slot + 1;
  }
  mul(x[1], y[1]);
  // no direct LDS load may land after the workgroup's LDS is handed on
  __builtin_amdgcn_s_waitcnt(0x0070);

  const int rbase = m0 + wm * FM * 32 + hi * 4;
  const int cbase = n0 + wn * FN * 32;
  if (part != nullptr) {  // a slice's sums go to its own [M][N] plane
    int* out = part + (size_t)slice * M * N;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int c = cbase + j * 32 + lr;
        if (c >= N) continue;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int m = rbase + i * 32 + (r >> 2) * 8 + (r & 3);
          if (m < M) out[(size_t)m * N + c] = acc[i][j][r];
        }
      }
    return;
  }
  const bool wide = epi_wide(ep, N) != 0;
  const rsrc_t rs = make_rsrc(sa, (uint32_t)M * 4u);  // M < 2^30
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    float s[16];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)((uint32_t)(rbase + i * 32 + g * 8) * 4u), 0, 0));
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

// Tiles of one kind (tm x tn), all of them once for each slice of kt_per_slice stages.
// Workgroups go to the eight XCDs (each with an L2 of its own) in turn.  These tiles, which the L2
// feeds, give each XCD a contiguous part of the work, in the order: slices, groups of eight tile
// rows, tile columns, rows of the group, so that the 32 tiles of an XCD at a time are about
// 8 x 4 (measured, 128 x 128 tiles: M = 1024, (4096, 4096) 32 -> 22 us, M = 512, (8192, 2048)
// 19 -> 15 us).
template <int WM, int WN, int FM, int FN, int NB>
__global__ __launch_bounds__(WM * WN * 64) void w8_ring_kernel(const int8_t* __restrict__ A, const float* __restrict__ sa,
                                                               const int8_t* __restrict__ W, const float* __restrict__ sw,
                                                               const Epi ep, int M, int N, int pitch, int tm, int tn,
                                                               int kt_per_slice, int* __restrict__ part) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int per_xcd = gridDim.x >> 3, left = gridDim.x & 7, xcd = blockIdx.x & 7;
  const int work = xcd * per_xcd + min(xcd, left) + (blockIdx.x >> 3);
  const int slice = work / (tm * tn), tile = work - slice * tm * tn;
  const int grp = tile / (8 * tn), in_grp = tile - grp * 8 * tn, rows_grp = min(8, tm - grp * 8);
  const int ti = grp * 8 + in_grp % rows_grp, tj = in_grp / rows_grp;
  ring_tile<WM, WN, FM, FN, NB>(smem, A, sa, W, sw, ep, M, N, pitch, ti * WM * FM * 32, tj * WN * FN * 32, slice,
                                kt_per_slice, part);
}

// The first `full` of tn column tiles in `high` 256-row tiles each, the columns left in `low`
// (FL 64)-row tiles.  In plain order: these tiles, bound by the matrix cores, are 2-3% faster so.
template <int FL>
__global__ __launch_bounds__(512) void w8_mixed_kernel(const int8_t* __restrict__ A, const float* __restrict__ sa,
                                                       const int8_t* __restrict__ W, const float* __restrict__ sw,
                                                       const Epi ep, int M, int N, int pitch, int full, int tn, int high,
                                                       int low, int kt_per_slice, int* __restrict__ part) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int n_high = full * high, n_all = n_high + (tn - full) * low;
  const int slice = blockIdx.x / (unsigned)n_all;
  const int tile = blockIdx.x - slice * n_all;
  if (tile < n_high) {
    ring_tile<2, 4, 4, 2, 2>(smem, A, sa, W, sw, ep, M, N, pitch, tile % high * 256, tile / high * 256, slice,
                             kt_per_slice, part);
  } else {
    const int t = tile - n_high;
    ring_tile<2, 4, FL, 2, 2>(smem, A, sa, W, sw, ep, M, N, pitch, t % low * FL * 64, (t / low + full) * 256, slice,
                              kt_per_slice, part);
  }
}

// Output = epilogue(sum of S int32 [M][N] planes), four columns a thread where rows of four
// are aligned (VEC: N a multiple of 4).
template <bool VEC>
__global__ __launch_bounds__(256) void w8_reduce_kernel(const int* __restrict__ part, int S, int M, int N,
                                                        const float* __restrict__ sa, const float* __restrict__ sw,
                                                        const Epi ep) {
  const size_t total = (size_t)M * N;
  constexpr int V = VEC ? 4 : 1;
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * V;
  if (i >= total) return;
  const int m = (int)(i / N), n = (int)(i - (size_t)m * N);
  if constexpr (VEC) {
    i32x4 v = *reinterpret_cast<const i32x4*>(part + i);
    for (int s = 1; s < S; ++s) v += *reinterpret_cast<const i32x4*>(part + s * total + i);
    float o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = w8_scaled(v[u], sa[m], sw[n + u]);
    if (epi_wide(ep, N) != 0) {
      epi_store4(epi_quad(ep, n, N), m, o);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) epi_put(ep, epi_col(ep, n + u), m, o[u]);
    }
  } else {
    int v = part[i];
    for (int s = 1; s < S; ++s) v += part[s * total + i];
    epi_put(ep, epi_col(ep, n), m, w8_scaled(v, sa[m], sw[n]));
  }
}

}  // namespace

namespace {

struct W8Plan {
  int tile = 0, full = 0, splits = 1;
};

// FL > 0: the 256 x 256 tiles mixed with (FL 64) x 256 ones.
template <int WM, int WN, int FM, int FN, int NB, int FL = 0>
hipError_t run_ring(const W8Args& a, const W8Plan& p, int* part, hipStream_t st) {
  static_assert(FL == 0 || (WM == 2 && WN == 4 && FM == 4 && FN == 2 && NB == 2), "w8_mixed_kernel's tile");
  constexpr int BM = WM * FM * 32, BN = WN * FN * 32, T = WM * WN * 64;
  constexpr int lds = NB * (BM + BN) * BK;
  const int M = (int)a.M, N = (int)a.N, pitch = (int)a.pitch;
  const int tm = (M + BM - 1) / BM, tn = (N + BN - 1) / BN;
  const int kt = (pitch + BK - 1) / BK;
  const int per = (kt + p.splits - 1) / p.splits;
  const int splits = (kt + per - 1) / per;  // every slice gets at least one stage
  if (splits == 1) part = nullptr;
  auto prepare = [](auto k) {
    if (lds <= 64 * 1024) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  };
  hipError_t e;
  if constexpr (FL > 0) {
    e = prepare(w8_mixed_kernel<FL>);
    if (e != hipSuccess) return e;
    const int low = (M + FL * 64 - 1) / (FL * 64);
    const int64_t wgs = ((int64_t)p.full * tm + (int64_t)(tn - p.full) * low) * splits;
    w8_mixed_kernel<FL><<<(unsigned)wgs, T, lds, st>>>(a.A, a.a_scales, a.W, a.w_scales, a.ep, M, N, pitch, p.full, tn, tm,
                                                       low, per, part);
  } else {
    e = prepare(w8_ring_kernel<WM, WN, FM, FN, NB>);
    if (e != hipSuccess) return e;
    w8_ring_kernel<WM, WN, FM, FN, NB><<<(unsigned)((int64_t)tm * tn * splits), T, lds, st>>>(
        a.A, a.a_scales, a.W, a.w_scales, a.ep, M, N, pitch, tm, tn, per, part);
  }
  e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const size_t total = (size_t)a.M * a.N;
  if (a.N % 4 == 0)
    w8_reduce_kernel<true><<<(unsigned)((total / 4 + 255) / 256), 256, 0, st>>>(part, splits, (int)a.M, (int)a.N, a.a_scales, a.w_scales, a.ep);
  else
    w8_reduce_kernel<false><<<(unsigned)((total + 255) / 256), 256, 0, st>>>(part, splits, (int)a.M, (int)a.N, a.a_scales, a.w_scales, a.ep);
  return hipGetLastError();
}

// Tiles, and what one stage of them takes, in us on MI355X (fitted to 33 sizes from
// (M, N, K) = (8, 4096, 4096) to (2048, 12288, 4096), where the plan is within 1% of the best of
// all tiles and splits): lat, the least time of a stage; mfma, a workgroup's share of the CU's
// matrix cores; bw, the LDS fill rate of the whole device in TB/s; and t0, a launch's start,
// first loads and stores.  bl: rows of the lower tiles that the 256-row ones are mixed with, and
// low: a stage of theirs.
struct Tile {
  const char* name;
  int bm, bn, slots;  // slots: workgroups that a CU's LDS holds
  double t0, lat, mfma, bw;
  int bl;
  double low;
};
constexpr Tile kTiles[] = {
    {"w8_256x256", 256, 256, 1, 8.0, 1.35, 1.81, 18.0, 192, 1.25},
    {"w8_256x256", 256, 256, 1, 8.0, 1.35, 1.81, 18.0, 128, 1.03},
    {"w8_256x128", 256, 128, 1, 6.5, 0.74, 1.02, 18.0, 0, 0.0},
    {"w8_128x128", 128, 128, 1, 5.5, 0.45, 0.56, 18.0, 0, 0.0},
    {"w8_128x64", 128, 64, 2, 4.7, 0.37, 0.33, 18.0, 0, 0.0},
    {"w8_64x64", 64, 64, 2, 4.3, 0.19, 0.23, 16.0, 0, 0.0},
};

// The plan with the least estimated time: rounds of workgroups, each the contraction's stages at
// the longest of the three figures above; a split adds a launch (4.5 us of the host's time) and
// the write and read of its int32 planes (8 TB/s: they fit the caches).  The 256 x 256 tiles take
// all of the columns, or those that make whole rounds, or none, and the lower tiles the others in
// a shorter last round (M = 3000, (8192, 2048) 62.9 -> 58.8 us, M = 2048, (11008, 4096)
// 100.5 -> 97.9; on weights from memory, six of them in turn, 77.7 -> 71.1 and 121.6 -> 123.5, and
// at M = 4096 208 -> 203.5).  The figures are those of calls on warm operands outside a graph; in
// a captured graph a split costs a launch's 2.5 us and not the host's 4.5.
W8Plan pick(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps, bool allow_split) {
  const int64_t cus = caps.cus > 0 ? caps.cus : 256, kt = ((K + 63) / 64 * 64 + BK - 1) / BK;
  W8Plan best;
  double best_t = 1e30;
  for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
    const Tile& c = kTiles[i];
    const int64_t rows = (M + c.bm - 1) / c.bm, tn = (N + c.bn - 1) / c.bn;
    for (int sp = 1; sp <= (allow_split ? 8 : 1); sp *= 2) {
      if (sp > 1 && kt / sp < 4) break;
      const int64_t steps = (kt + sp - 1) / sp;
      for (const int64_t full : {tn, rows * tn / cus * cus / rows, (int64_t)0}) {
        if (full < tn && c.bl == 0) break;
        const int64_t wgs = rows * full * sp;
        const int64_t rounds = (wgs + cus * c.slots - 1) / (cus * c.slots);
        // workgroups of the fullest CU; a round that leaves CUs idle runs at a higher clock
        const int64_t resident = std::min(wgs, cus * c.slots);
        const double per_cu = resident <= cus ? (double)resident / cus : (double)((resident + cus - 1) / cus);
        const double fill = (double)resident * (c.bm + c.bn) * BK / c.bw * 1e-6;
        const double stage = std::max(std::max(c.lat, c.mfma * per_cu), fill);
        const int64_t lows = full < tn ? (tn - full) * ((M + c.bl - 1) / c.bl) * sp : 0;
        const double t = c.t0 + rounds * steps * stage + (double)((lows + cus - 1) / cus * steps) * c.low +
                         (sp > 1 ? 4.5 + sp * M * N * 8.0 / 8.0 * 1e-6 : 0.0);
        if (t < best_t) {
          best_t = t;
          best = W8Plan{i, (int)full, sp};
        }
      }
    }
  }
  return best;
}

size_t plan_bytes(int64_t M, int64_t N, const W8Plan& p) { return p.splits > 1 ? (size_t)p.splits * M * N * 4 : 0; }

}  // namespace

size_t w8_mm_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps) {
  return w8_decode_supported(M) ? 0 : plan_bytes(M, N, pick(M, N, K, caps, true));
}

const char* w8_mm_name(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps) {
  static thread_local char buf[48];
  if (w8_decode_supported(M)) return "w8_decode";
  const W8Plan p = pick(M, N, K, caps, true);
  const Tile& c = kTiles[p.tile];
  int at = snprintf(buf, sizeof(buf), "%s", c.name);
  if (p.full < (N + c.bn - 1) / c.bn) at += snprintf(buf + at, sizeof(buf) - at, "+%dx256", c.bl);
  if (p.splits > 1) snprintf(buf + at, sizeof(buf) - at, "_splitk%d", p.splits);
  return buf;
}

hipError_t launch_w8_mm(const W8Args& a, const DeviceCaps& caps, void* ws, size_t ws_bytes, hipStream_t st) {
  if (w8_decode_supported(a.M)) return launch_w8_decode(a, caps, st);
  W8Plan p = pick(a.M, a.N, a.K, caps, true);
  if (plan_bytes(a.M, a.N, p) > ws_bytes) p = pick(a.M, a.N, a.K, caps, false);
  int* part = static_cast<int*>(ws);
  switch (p.tile) {
    case 0: return run_ring<2, 4, 4, 2, 2, 3>(a, p, part, st);
    case 1: return run_ring<2, 4, 4, 2, 2, 2>(a, p, part, st);
    case 2: return run_ring<4, 2, 2, 2, 3>(a, p, part, st);
    case 3: return run_ring<4, 2, 1, 2, 3>(a, p, part, st);
    case 4: return run_ring<2, 2, 2, 1, 3>(a, p, part, st);
    default: return run_ring<2, 2, 1, 1, 4>(a, p, part, st);
  }
}

}  // namespace w4
