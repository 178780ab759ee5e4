// Product of microscaled 4-bit rows on the matrix cores, for gfx950:
//   Y[m][n] = out_rne(sum_k a[m][k] w[n][k] + bias[n]),  a = code * 2^(exponent - 127), w likewise,
// products exact, sums in fp32.
#include <algorithm>
#include <cstdio>
#include <type_traits>

#include "api_common.h"
#include "epilogue.h"
#include "launch.h"
#include "mx.h"

namespace w4 {

namespace {

constexpr int BK = 128;  // contraction bytes of a stage: 256 columns, a 128-byte line of each row

// Words of exponents that each of T threads loads in a stage of `rows` rows, and a stage's bytes of LDS.
constexpr int exponent_loads(int T, int rows) { return (rows * 2 + T - 1) / T; }
constexpr int stage_bytes(int T, int rows) { return rows * BK + exponent_loads(T, rows) * T * 4; }

// One workgroup of WM x WN waves computes a (WM FM 32) x (WN FN 32) tile.  Both operands run along
// the contraction, so a stage (256 columns of every row of both tiles and their eight exponents a
// row) goes global -> LDS with direct loads, through a ring of NB stages.  A stage's code rows are
// 128 bytes, their 16-byte chunk index XOR-ed with (row / 2) % 8 on the source address, so that the
// 16-byte LDS reads of 32 rows hit distinct banks.
// v_mfma_scale_f32_32x32x64_f8f6f4: lane l supplies a block of 32 columns of row l % 32 of each
// operand (columns 32 (l / 32) ..) with its exponent, one byte of a register, and holds column
// l % 32 of the result, register r being row 8 (r / 4) + 4 (l / 32) + (r % 4).  Product p of a
// stage's four takes exponents 2p + l / 32 of the row: bytes 0 and 2 of the two words, the words
// of the upper half of the wave moved down by a byte.
// The one barrier a stage says that the stage has landed for every wave, and that every wave has
// read the stage before it, whose slot the direct loads of this stage then fill.  The stage's
// first operands are read behind the barrier while the last products of the stage before run.
// What bounds it: a 256 x 256 tile's stage takes 1.8 us, of which its products alone 1.3 and its loads and
// LDS reads alone 1.5; behind that, a round of tiles stores its results while nothing multiplies (10 of
// 84 us at (M, N, K) = (4096, 8192, 4096)).  8192^3: 3.65 PFLOP/s (zeros 4.5: the clock gives way to
// random operands), (4096, 11008, 4096) 111 us, 3.3 PFLOP/s.  Exponents loaded for two or four stages at a
// time, and a stage ahead of their codes, were within 2% of this, either way.
template <int WM, int WN, int FM, int FN, int NB>
__device__ __forceinline__ void ring_tile(char* smem, const uint8_t* __restrict__ A, const uint8_t* __restrict__ ae,
                                          const uint8_t* __restrict__ W, const uint8_t* __restrict__ we, const Epi& ep, int M,
                                          int N, int pitch, int m0, int n0, int slice, int kt_per_slice,
                                          float* __restrict__ part) {
  constexpr int T = WM * WN * 64, BM = WM * FM * 32, BN = WN * FN * 32;
  constexpr int CH = BK / 16, UA = BM * CH / T, UB = BN * CH / T;  // chunks a thread loads of each tile in a stage
  constexpr int UE = exponent_loads(T, BM + BN);   // words of exponents: two of each row
  constexpr int OE = (BM + BN) * BK, STAGE = stage_bytes(T, BM + BN);
  constexpr int UL = UA + UB + UE;
  auto swz = [](int row) { return (row >> 1) & 7; };
  static_assert(BM * CH % T == 0 && BN * CH % T == 0 && BM % 32 == 0 && BN % 32 == 0, "tile split");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int epitch = pitch >> 4;  // exponents of a row (bytes)
  const rsrc_t ra = mx_rsrc(A + (size_t)m0 * pitch, (uint32_t)min(BM, M - m0) * (uint32_t)pitch);
  const rsrc_t rb = mx_rsrc(W + (size_t)n0 * pitch, (uint32_t)min(BN, N - n0) * (uint32_t)pitch);
  const uint8_t* ea0 = ae + (size_t)m0 * epitch;
  const uint8_t* eb0 = we + (size_t)n0 * epitch;
  const uint32_t ea_bytes = (uint32_t)min(BM, M - m0) * (uint32_t)epitch, eb_bytes = (uint32_t)min(BN, N - n0) * (uint32_t)epitch;
  int oa[UA], ob[UB], oe[UE];
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
  // word u of the exponents: row u / 2 of the first tile, then of the second; a wave's 64 words are of
  // one tile, and past both they have an empty resource
#pragma unroll
  for (int i = 0; i < UE; ++i) {
    const int u = tid + i * T;
    oe[i] = ((u < BM * 2 ? u : u - BM * 2) >> 1) * epitch + ((tid & 1) << 2);
  }
  // this slice's stages
  const int k0 = slice * kt_per_slice;
  const int KT = min((pitch + BK - 1) / BK - k0, kt_per_slice);
  // loads [lo, hi) of stage kt into ring slot `slot`; past the end the last stage again, never read
  auto dma_part = [&](int kt, int slot, int lo, int hi) {
    const int st = k0 + min(kt, KT - 1), so = st * BK, se = st * 8;
    char* base = smem + slot * STAGE + wave * 1024;
    char* ebase = smem + slot * STAGE + OE + wave * 256;
#pragma unroll
    for (int i = 0; i < UL; ++i) {
      if (i < lo || i >= hi) continue;
      if (i < UA)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(base + i * T * 16), 16, (int)oa[i < UA ? i : 0], (int)so, 0, 0);
      else if (i < UA + UB)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(base + BM * BK + (i - UA) * T * 16), 16,
                                                 (int)ob[i >= UA && i < UA + UB ? i - UA : 0], (int)so, 0, 0);
      else {
        const int u = wave * 64 + (i - UA - UB) * T;
        const rsrc_t re = mx_rsrc(u < BM * 2 ? ea0 : eb0, u < BM * 2 ? ea_bytes : u < (BM + BN) * 2 ? eb_bytes : 0u);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(re, (lds_void*)(ebase + (i - UA - UB) * T * 4), 4,
                                                 (int)oe[i >= UA + UB ? i - UA - UB : 0], (int)se, 0, 0);
      }
    }
  };
  // all but the last NB - 2 stages landed and this wave's reads done, then a barrier with no fence
  // (a fence would wait for every load in flight)
  auto sync = [&]() {
    constexpr int n = (NB - 2) * UL;
    static_assert(n < 64, "the wait's counter");
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
  const int ga = OE + (wm * FM * 32 + lr) * 8, gb = OE + BM * 8 + (wn * FN * 32 + lr) * 8;
  const int down = hi * 8;
  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  u32x4 x[2][FM], y[2][FN];
  uint32_t ex[2][FM], ey[2][FN];    // a stage's exponents: products 0 and 1, 2 and 3
  uint32_t lx[FM], ly[FN];          // those of the product that is still to come from the stage before
  auto read_x = [&](const char* base, int kk, u32x4 (&v)[FM]) {
#pragma unroll
    for (int i = 0; i < FM; ++i) v[i] = *reinterpret_cast<const u32x4*>(base + (fa ^ (kk * 32)) + i * 32 * BK);
  };
  auto read_y = [&](const char* base, int kk, u32x4 (&v)[FN]) {
#pragma unroll
    for (int j = 0; j < FN; ++j) v[j] = *reinterpret_cast<const u32x4*>(base + (fb ^ (kk * 32)) + j * 32 * BK);
  };
  auto mul1 = [&](auto byte, const u32x4& a, uint32_t ea, const u32x4& b, uint32_t eb, f32x16& c) {
    constexpr int B = decltype(byte)::value;
    c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, kFp4, kFp4, B, (int)ea, B, (int)eb);
  };
  auto mul = [&](auto byte, const u32x4 (&a)[FM], const uint32_t (&ea)[FM], const u32x4 (&b)[FN], const uint32_t (&eb)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) mul1(byte, a[i], ea[i], b[j], eb[j], acc[i][j]);
  };
  const std::integral_constant<int, 0> b0;
  const std::integral_constant<int, 2> b2;
#pragma unroll
  for (int k = 0; k < NB - 1; ++k) dma_part(k, k, 0, UL);
  int slot = 0;
  for (int kt = 0; kt < KT; ++kt) {
    sync();
    const char* base = smem + slot * STAGE;
    const int free_slot = slot == 0 ? NB - 1 : slot - 1;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const u32x2 e = *reinterpret_cast<const u32x2*>(base + ga + i * 32 * 8);
      ex[0][i] = e[0];
      ex[1][i] = e[1];
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const u32x2 e = *reinterpret_cast<const u32x2*>(base + gb + j * 32 * 8);
      ey[0][j] = e[0];
      ey[1][j] = e[1];
    }
    read_x(base, 0, x[0]);
    read_y(base, 0, y[0]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      // the last products of the stage before, their registers refilled one by one
      if (kt > 0) {
#pragma unroll
        for (int j = 0; j < FN; ++j) mul1(b2, x[1][i], lx[i], y[1][j], ly[j], acc[i][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
      dma_part(kt + NB - 1, free_slot, i * UL / FM, (i + 1) * UL / FM);
      x[1][i] = *reinterpret_cast<const u32x4*>(base + (fa ^ 32) + i * 32 * BK);
      __builtin_amdgcn_sched_barrier(0);
    }
    read_y(base, 1, y[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < FM; ++i) ex[h][i] >>= down;
#pragma unroll
      for (int j = 0; j < FN; ++j) ey[h][j] >>= down;
    }
    __builtin_amdgcn_sched_barrier(0);
    mul(b0, x[0], ex[0], y[0], ey[0]);
    const bool whole = (k0 + kt) * BK + 64 < pitch;  // the row's last stage may be half a one
    if (whole) {
      __builtin_amdgcn_sched_barrier(0);
      read_x(base, 2, x[0]);
      read_y(base, 2, y[0]);
      __builtin_amdgcn_sched_barrier(0);
      mul(b2, x[1], ex[0], y[1], ey[0]);
      __builtin_amdgcn_sched_barrier(0);
      read_x(base, 3, x[1]);
      read_y(base, 3, y[1]);
      __builtin_amdgcn_sched_barrier(0);
      mul(b0, x[0], ex[1], y[0], ey[1]);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) lx[i] = whole ? ex[1][i] : ex[0][i];
#pragma unroll
    for (int j = 0; j < FN; ++j) ly[j] = whole ? ey[1][j] : ey[0][j];
    slot = slot == NB - 1 ? 0 : slot + 1;
  }
  mul(b2, x[1], lx, y[1], ly);
  // no direct LDS load may land after the workgroup's LDS is handed on
  __builtin_amdgcn_s_waitcnt(0x0070);

  const int rbase = m0 + wm * FM * 32 + hi * 4;
  const int cbase = n0 + wn * FN * 32;
  if (part != nullptr) {  // a slice's sums go to its own [M][N] plane
    float* out = part + (size_t)slice * M * N;
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
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int c = cbase + j * 32 + lr;
    if (wide) {
      const EpiQuad q = epi_quad(ep, cbase + j * 32 + (lr & ~3), N);
#pragma unroll
      for (int i = 0; i < FM; ++i) epi_put_block_wide(q, acc[i][j], rbase + i * 32, M, lane);
    } else if (c < N) {
      const EpiCol col = epi_col(ep, c);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int m = rbase + i * 32 + (r >> 2) * 8 + (r & 3);
          if (m < M) epi_put(ep, col, m, acc[i][j][r]);
        }
    }
  }
}

// Work of a launch: the first `full` column tiles in (WM FB 32)-row tiles, the columns left in
// (WM FM 32)-row tiles; all of that once for each slice of the contraction.
struct Grid {
  int full, tn;   // column tiles of the first kind, and in all
  int high, low;  // row tiles of the two kinds
  int per;        // stages of a slice
};

// Workgroups go to the eight XCDs (each with an L2 of its own) in turn; of each kind of tile an XCD gets
// a contiguous part, in the order: groups of eight tile rows, tile columns, rows of the group, so that
// its 32 tiles at a time are about 8 x 4 (against plain order, at 8192^3 301 us, 320 without; M = 512,
// (8192, 2048) 12.4, 14.1).
template <int WM, int WN, int FB, int FM, int FN, int NB>
__global__ __launch_bounds__(WM * WN * 64) void mx_ring_kernel(const uint8_t* __restrict__ A, const uint8_t* __restrict__ ae,
                                                               const uint8_t* __restrict__ W, const uint8_t* __restrict__ we,
                                                               const Epi ep, int M, int N, int pitch, const Grid g,
                                                               float* __restrict__ part) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int n_high = FB > 0 ? g.full * g.high : 0, n_all = n_high + (g.tn - g.full) * g.low;
  const int slice = blockIdx.x / (unsigned)n_all;
  int at = blockIdx.x - (unsigned)slice * n_all;
  const bool high = at < n_high;
  if (!high) at -= n_high;
  const int kind = high ? n_high : n_all - n_high, rows = high ? g.high : g.low, cols = high ? g.full : g.tn - g.full;
  const int per_xcd = kind >> 3, left = kind & 7, xcd = at & 7;
  const int tile = xcd * per_xcd + min(xcd, left) + (at >> 3);
  const int grp = tile / (8 * cols), in_grp = tile - grp * 8 * cols, rows_grp = min(8, rows - grp * 8);
  const int tr = grp * 8 + in_grp % rows_grp, tc = in_grp / rows_grp + (high ? 0 : g.full);
  if constexpr (FB > 0)
    if (high) {
      ring_tile<WM, WN, FB, FN, NB>(smem, A, ae, W, we, ep, M, N, pitch, tr * WM * FB * 32, tc * WN * FN * 32, slice, g.per, part);
      return;
    }
  ring_tile<WM, WN, FM, FN, NB>(smem, A, ae, W, we, ep, M, N, pitch, tr * WM * FM * 32, tc * WN * FN * 32, slice, g.per, part);
}

struct MxPlan {
  int tile = 0, full = 0, splits = 1;
};

template <int WM, int WN, int FB, int FM, int FN, int NB>
hipError_t run_ring(const MxArgs& a, const MxPlan& p, float* part, hipStream_t st) {
  constexpr int BM = WM * FM * 32, BN = WN * FN * 32, T = WM * WN * 64, BH = FB > 0 ? WM * FB * 32 : 1;
  const int lds = NB * stage_bytes(T, (p.full > 0 ? BH : BM) + BN);
  const int M = (int)a.M, N = (int)a.N, pitch = (int)(a.P / 2);
  const int kt = (pitch + BK - 1) / BK;
  Grid g = {};
  g.tn = (N + BN - 1) / BN;
  g.full = p.full;
  g.high = FB > 0 ? (M + BH - 1) / BH : 0;
  g.low = (M + BM - 1) / BM;
  g.per = (kt + p.splits - 1) / p.splits;
  const int splits = (kt + g.per - 1) / g.per;  // every slice gets at least one stage
  auto k = mx_ring_kernel<WM, WN, FB, FM, FN, NB>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int64_t wgs = ((int64_t)g.full * g.high + (int64_t)(g.tn - g.full) * g.low) * splits;
  k<<<(unsigned)wgs, T, lds, st>>>(a.A, a.a_scales, a.W, a.w_scales, a.ep, M, N, pitch, g, splits > 1 ? part : nullptr);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  return launch_splitk_reduce(part, splits, a.M, 0, a.N, a.ep, st);
}

// Tiles of bm (0: none) and lower rows and bn columns, and what one stage of them takes, in us on MI355X
// (fitted to 20 sizes from (M, N, K) = (32, 2048, 2048) to (4096, 11008, 4096), in a captured graph, where
// the plan is within 1% of the best of all tiles and splits; of 32 tokens and fewer only long rows of few
// channels come here now):
// high, of a bm-row tile; lat, the least time of a stage of a lower one; mfma, a workgroup's share of
// the CU's matrix cores; and t0, a launch's start, first loads and stores.
struct Tile {
  const char* name;
  int bm, low, bn, slots;  // slots: workgroups that a CU's LDS holds
  double t0, high, lat, mfma;
};
constexpr Tile kTiles[] = {
    {"mx4_256x256", 256, 192, 256, 1, 4.9, 2.20, 1.57, 1.72},
    {"mx4_256x256", 256, 128, 256, 1, 4.9, 2.20, 1.23, 1.47},
    {"mx4_256x128", 0, 256, 128, 1, 6.75, 0.00, 0.87, 1.31},
    {"mx4_128x128", 0, 128, 128, 1, 6.25, 0.00, 0.62, 0.81},
    {"mx4_128x64", 0, 128, 64, 2, 5.3, 0.00, 0.37, 0.45},
    {"mx4_64x64", 0, 64, 64, 2, 4.7, 0.00, 0.24, 0.29},
};

// The plan with the least estimated time: rounds of workgroups, each the contraction's stages; a split
// adds a launch and the write and read of its fp32 planes.  256 x 256 tiles take all of the columns,
// those that make whole rounds, or none, and the lower tiles the others in a shorter last round.
MxPlan pick(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps, bool allow_split) {
  const int64_t cus = caps.cus > 0 ? caps.cus : 256, kt = (mx_pitch(K) / 2 + BK - 1) / BK;
  MxPlan best;
  double best_t = 1e30;
  for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
    const Tile& c = kTiles[i];
    const int64_t low = (M + c.low - 1) / c.low, high = c.bm > 0 ? (M + c.bm - 1) / c.bm : 0, tn = (N + c.bn - 1) / c.bn;
    for (int sp = 1; sp <= (allow_split ? 8 : 1); sp *= 2) {
      if (sp > 1 && kt / sp < 4) break;
      const int64_t steps = (kt + sp - 1) / sp;
      for (const int64_t full : {(int64_t)0, high > 0 ? high * tn / cus * cus / high : 0, high > 0 ? tn : 0}) {
        const int64_t a = full * high * sp, b = (tn - full) * low * sp;
        const int64_t rounds = (b + cus * c.slots - 1) / (cus * c.slots);
        // workgroups of the fullest CU; a round that leaves CUs idle runs at a higher clock
        const int64_t resident = std::min(b, cus * c.slots);
        const double per_cu = resident <= cus ? (double)resident / cus : (double)((resident + cus - 1) / cus);
        const double t = c.t0 + (double)((a + cus - 1) / cus * steps) * c.high +
                         (double)(rounds * steps) * std::max(c.lat, c.mfma * per_cu) +
                         (sp > 1 ? 2.1 + sp * M * N * 8.0 / 8.0 * 1e-6 : 0.0);
        if (t < best_t) {
          best_t = t;
          best = MxPlan{i, (int)full, sp};
        }
      }
    }
  }
  return best;
}

size_t plan_bytes(int64_t M, int64_t N, const MxPlan& p) { return p.splits > 1 ? (size_t)p.splits * M * N * 4 : 0; }

}  // namespace

size_t mx_mm_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps) {
  return mx_few_supported(M, N, K, caps) || mx_decode_ready_supported(M, K) ? 0 : plan_bytes(M, N, pick(M, N, K, caps, true));
}

const char* mx_mm_name(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps) {
  static thread_local char buf[48];
  if (mx_few_supported(M, N, K, caps)) return "mx4_few";
  if (mx_decode_ready_supported(M, K)) return "mx4_decode";
  const MxPlan p = pick(M, N, K, caps, true);
  const Tile& c = kTiles[p.tile];
  int at = snprintf(buf, sizeof(buf), "%s", c.name);
  if (c.bm > 0 && p.full < (N + c.bn - 1) / c.bn) at += snprintf(buf + at, sizeof(buf) - at, "+%dx256", c.low);
  if (p.splits > 1) snprintf(buf + at, sizeof(buf) - at, "_splitk%d", p.splits);
  return buf;
}

hipError_t launch_mx_mm(const MxArgs& a, const DeviceCaps& caps, void* ws, size_t ws_bytes, hipStream_t st) {
  if (mx_few_supported(a.M, a.N, a.K, caps)) return launch_mx_few(a, caps, st);
  if (mx_decode_ready_supported(a.M, a.K)) return launch_mx_decode(a, caps, st);
  MxPlan p = pick(a.M, a.N, a.K, caps, true);
  if (plan_bytes(a.M, a.N, p) > ws_bytes) p = pick(a.M, a.N, a.K, caps, false);
  float* part = static_cast<float*>(ws);
  switch (p.tile) {
    case 0: return run_ring<2, 4, 4, 3, 2, 2>(a, p, part, st);
    case 1: return run_ring<2, 4, 4, 2, 2, 2>(a, p, part, st);
    case 2: return run_ring<4, 2, 0, 2, 2, 3>(a, p, part, st);
    case 3: return run_ring<2, 2, 0, 2, 2, 4>(a, p, part, st);
    case 4: return run_ring<2, 2, 0, 2, 1, 3>(a, p, part, st);
    default: return run_ring<2, 2, 0, 1, 1, 4>(a, p, part, st);
  }
}

}  // namespace w4
