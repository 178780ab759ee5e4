// Input gradient of the microscaled 4-bit product (mx4_mm_t), for gfx950:
//   dX[m][k] = out_rne(sum_n dY[m][n] w[n][k]),  w = code * 2^(exponent - 127),
// fp32 accumulation.  The contraction runs across the weight's rows, along which the exponents
// change with every row, so the 4-bit matrix instructions do not apply; but w has two significant
// bits, so bf16 holds it exactly, and dY enters as bf16 parts whose sum it is (one of bf16, two of
// fp16, three of fp32): the parts lengthen the contraction, and nothing is rounded before the sums.
// What bounds it: the bf16 matrix cores, at the clock that they leave, and the last, partial round of tiles.
// (M, N, K) = (2048, 4096, 8192), whole rounds: 110 us, 1.25 PFLOP/s (the library's product on a weight that
// is bf16 already: 101); (2048, 4096, 11008), 1.34 rounds: 167, 1.11 PFLOP/s.
#include <algorithm>

#include "api_common.h"
#include "epilogue.h"
#include "launch.h"
#include "mx.h"

namespace w4 {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int BK = 64;  // contraction rows of a stage

constexpr int stage_bytes(int bm, int bn) { return bm * 128 + BK * bn * 2; }

// One workgroup of WM x WN waves computes a (WM FM 32) x (WN FN 32) tile.  A stage is 64 columns of
// dY's rows and 64 rows of the weight, in one of two places in LDS.  Both go through registers, read one
// stage ahead: the weight's blocks of 32 columns (16 bytes and their exponent) are widened once in the
// workgroup on the way, and behind direct loads of dY the compiler would wait for all of them ahead of
// every transposing read.
//   dY's rows of 128 bytes have their 16-byte chunk index XOR-ed with (row / 2) % 8.  The weight's rows
//   are bf16: a row's 64-byte pieces (a block) at piece ^ (row % 4), a piece's 16-byte quarters at
//   quarter ^ (piece / 4 % 2 + 2 (row % 2)).  Sixteen lanes' writes, and the 4-row reads of half a
//   wave, then hit distinct banks.
//   v_mfma_f32_32x32x16_bf16: lane l supplies dY row l % 32 and weight column l % 32, contraction
//   slots 8 (l / 32) .. + 7 of 16.  A transposing read takes sixteen lanes to 4 rows of 16 columns
//   and returns lane l column l of the four rows; two make an operand.
// The one barrier a stage says that it is written, and that the stage before it has been read, whose
// place the writes of the stage after it then fill.  The operands of product p + 1 are read while
// product p of a stage's four runs; the last one runs behind the next stage's barrier.
template <int WM, int WN, int FM, int FN>
__device__ __forceinline__ void grad_tile(char* smem, const uint16_t* __restrict__ dY, const uint8_t* __restrict__ W,
                                          const uint8_t* __restrict__ we, const Epi& ep, int M, int N, int L, int K, int ld,
                                          int parts, int P, int m0, int c0, int slice, int per, float* __restrict__ part) {
  constexpr int T = WM * WN * 64, BM = WM * FM * 32, BN = WN * FN * 32;
  constexpr int CB = BN / 32, UA = BM * 8 / T, UB = BK * CB / T;  // chunks a thread loads in a stage
  static_assert(BM * 8 % T == 0 && BK * CB % T == 0 && (CB & (CB - 1)) == 0 && CB >= 4, "tile split");
  constexpr int OW = BM * 128, STAGE = stage_bytes(BM, BN);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int row = P >> 1, erow = P >> 5;
  const int nst = (N + BK - 1) / BK;  // stages of a part
  const int k0 = slice * per, KT = min(nst * parts - k0, per);
  int oa[UA], ca[UA], ob[UB], oe[UB], at_a[UA], at_w[UB];
#pragma unroll
  for (int i = 0; i < UA; ++i) {
    const int u = tid + i * T, r = u >> 3;
    ca[i] = (u & 7) * 8;
    oa[i] = (r * parts * ld + ca[i]) * 2;
    at_a[i] = r * 128 + (((u & 7) ^ ((r >> 1) & 7)) << 4);
  }
#pragma unroll
  for (int i = 0; i < UB; ++i) {
    const int u = tid + i * T, r = u / CB, c = u % CB;
    ob[i] = r * row + (c0 >> 1) + c * 16;
    oe[i] = r * erow + (c0 >> 5) + c;
    at_w[i] = OW + r * (BN * 2) + ((c ^ (r & 3)) << 6) + ((((c >> 2) & 1) | (r & 1) << 1) << 4);
  }
  const uint32_t a_bytes = (uint32_t)min(BM, M - m0) * (uint32_t)(parts * ld) * 2u;
  u32x4 ar[UA], wr[UB];
  uint32_t er[UB];
  // stage kt (past the end the last one again, never used)
  auto load = [&](int kt) {
    const int s = k0 + min(kt, KT - 1), pt = s / nst, n0 = (s - pt * nst) * BK;
    const uint32_t skip = (uint32_t)(pt * ld + n0), rows = (uint32_t)min(BK, N - n0);
    // columns past the last one are asked for out of range and so 0
    const rsrc_t ra = mx_rsrc(dY + (size_t)m0 * parts * ld + skip, a_bytes - skip * 2u);
    const rsrc_t rb = mx_rsrc(W + (size_t)n0 * row, rows * (uint32_t)row);
    const rsrc_t re = mx_rsrc(we + (size_t)n0 * erow, rows * (uint32_t)erow);
#pragma unroll
    for (int i = 0; i < UB; ++i) {
      wr[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rb, ob[i], 0, 0));
      er[i] = __builtin_amdgcn_raw_buffer_load_b8(re, oe[i], 0, 0);
    }
#pragma unroll
    for (int i = 0; i < UA; ++i)
      ar[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, n0 + ca[i] < L ? oa[i] : 0x7FFFFFFF, 0, 0));
  };
  auto put_w = [&](int place) {
#pragma unroll
    for (int i = 0; i < UB; ++i) {
      const float p = __uint_as_float(er[i] << 23);  // (its exponent bits count alone)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<u32x4*>(smem + ((at_w[i] + place * STAGE) ^ (q << 4))) = mx_bf16x8(wr[i][q], p);
    }
  };
  auto put_a = [&](int place) {
#pragma unroll
    for (int i = 0; i < UA; ++i) *reinterpret_cast<u32x4*>(smem + at_a[i] + place * STAGE) = ar[i];
  };
  // this wave's LDS reads and writes done, then a barrier with no fence (a fence would wait for the
  // loads in flight)
  auto sync = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  const int lr = lane & 31, hi = lane >> 5;
  const int fa = (wm * FM * 32 + lr) * 128 + ((hi ^ ((lr >> 1) & 7)) << 4);  // product p at ^ 32 p
  // transposed operand: rows 16 p + 8 hi + 4 h + r4, this lane's 8 bytes of them
  const int r4 = (lane & 15) >> 2, quarter = ((lane >> 4) & 1) * 2 + ((lane >> 1) & 1);
  int fb[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int c = wn * FN + j;
    fb[j] = OW + (8 * hi + r4) * (BN * 2) + ((c ^ r4) << 6) + ((quarter ^ (((c >> 2) & 1) | (r4 & 1) << 1)) << 4) + (lane & 1) * 8;
  }
  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  u32x4 x[2][FM], y[2][FN];
  auto read = [&](char* base, int p, u32x4 (&v)[FM], u32x4 (&w)[FN]) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      u32x2 h[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        h[k] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + fb[j] + (16 * p + 4 * k) * (BN * 2))));
      w[j] = u32x4{h[0][0], h[0][1], h[1][0], h[1][1]};
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) v[i] = *reinterpret_cast<const u32x4*>(base + (fa ^ (32 * p)) + i * 32 * 128);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mul = [&](const u32x4 (&v)[FM], const u32x4 (&w)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma_op<false>(v[i], w[j], acc[i][j]);
  };

  load(0);
  put_w(0);
  put_a(0);
  load(1);
  for (int kt = 0; kt < KT; ++kt) {
    sync();
    char* base = smem + (kt & 1) * STAGE;
    const int other = (kt + 1) & 1;
    read(base, 0, x[0], y[0]);
    if (kt > 0) mul(x[1], y[1]);
    __builtin_amdgcn_sched_barrier(0);
    read(base, 1, x[1], y[1]);
    mul(x[0], y[0]);
    put_w(other);
    __builtin_amdgcn_sched_barrier(0);
    read(base, 2, x[0], y[0]);
    mul(x[1], y[1]);
    put_a(other);
    __builtin_amdgcn_sched_barrier(0);
    load(kt + 2);
    read(base, 3, x[1], y[1]);
    mul(x[0], y[0]);
  }
  mul(x[1], y[1]);
  const int cbase = c0 + wn * FN * 32, mbase = m0 + wm * FM * 32 + hi * 4;
  const bool wide = part == nullptr && epi_wide(ep, K) != 0;
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int c = cbase + j * 32 + lr;
    if (wide) {
      const EpiQuad q = epi_quad(ep, cbase + j * 32 + (lr & ~3), K);
#pragma unroll
      for (int i = 0; i < FM; ++i) epi_put_block_wide(q, acc[i][j], mbase + i * 32, M, lane);
      continue;
    }
    if (c >= K) continue;
    if (part != nullptr) {  // a slice's sums go to its own [M][K] plane
      float* out = part + (size_t)slice * M * K + c;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int m = mbase + i * 32 + (r >> 2) * 8 + (r & 3);
          if (m < M) out[(size_t)m * K] = acc[i][j][r];
        }
      continue;
    }
    const EpiCol col = epi_col(ep, c);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = mbase + i * 32 + (r >> 2) * 8 + (r & 3);
        if (m < M) epi_put(ep, col, m, acc[i][j][r]);
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

// Workgroups go to the eight XCDs in turn; of each kind of tile an XCD gets a contiguous part, in the
// order: groups of eight tile rows, tile columns, rows of the group.
template <int WM, int WN, int FB, int FM, int FN>
__global__ __launch_bounds__(WM * WN * 64) void mx_grad_kernel(const uint16_t* __restrict__ dY, const uint8_t* __restrict__ W,
                                                               const uint8_t* __restrict__ we, const Epi ep, int M, int N, int L,
                                                               int K, int ld, int parts, int P, const Grid g,
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
      grad_tile<WM, WN, FB, FN>(smem, dY, W, we, ep, M, N, L, K, ld, parts, P, tr * WM * FB * 32, tc * WN * FN * 32, slice, g.per,
                                part);
      return;
    }
  grad_tile<WM, WN, FM, FN>(smem, dY, W, we, ep, M, N, L, K, ld, parts, P, tr * WM * FM * 32, tc * WN * FN * 32, slice, g.per, part);
}

// Tiles of bm (0: none) and lower rows and bn columns, and what one stage of them takes, in us on MI355X
// (fitted to 17 sizes from (M, N, K) = (32, 4096, 4096) to (4096, 4096, 11008), in a captured graph, where
// the plan is within 1% of the best of all tiles and splits):
// high, of a bm-row tile; lat, the least time of a stage of a lower one; mfma, a workgroup's share of
// the CU's matrix cores; and t0, a launch's start, first loads and stores.
struct Tile {
  int bm, low, bn, slots;  // slots: workgroups that a CU's LDS holds
  double t0, high, lat, mfma;
};
constexpr Tile kTiles[] = {
    {256, 128, 256, 1, 9.3, 1.53, 0.84, 0.91},
    {0, 128, 128, 2, 10.5, 0.00, 0.60, 0.49},
    {0, 64, 128, 3, 10.1, 0.00, 0.41, 0.29},
    {0, 32, 128, 4, 9.9, 0.00, 0.31, 0.21},
};

struct GradPlan {
  int tile = 0, full = 0, splits = 1;
};

// The plan with the least estimated time: rounds of workgroups, each the contraction's stages; a split
// adds the write and read of its planes (and a launch, most of which the fit found in t0).  256-row tiles
// take none of the columns, all, or those that make whole rounds, the last, partial round then being one
// of 128-row tiles.
GradPlan pick(int64_t M, int64_t N, int64_t K, int parts, const DeviceCaps& caps, bool allow_split) {
  const int64_t cus = caps.cus > 0 ? caps.cus : 256, kt = (N + BK - 1) / BK * parts;
  GradPlan best;
  double best_t = 1e30;
  for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
    const Tile& c = kTiles[i];
    const int64_t tn = (K + c.bn - 1) / c.bn, low = (M + c.low - 1) / c.low;
    const int64_t high = c.bm > 0 ? (M + c.bm - 1) / c.bm : 0;
    for (int sp = 1; sp <= (allow_split ? 8 : 1); sp *= 2) {
      if (sp > 1 && kt / sp < 4) break;
      const int64_t steps = (kt + sp - 1) / sp;
      const int64_t some = high > 0 ? high * tn / cus * cus / high : 0;
      for (const int64_t full : {(int64_t)0, some, high > 0 ? tn : 0}) {
        const int64_t a = full * high * sp, b = (tn - full) * low * sp;
        const int64_t rounds = (b + cus * c.slots - 1) / (cus * c.slots);
        // workgroups of the fullest CU; a round that leaves CUs idle runs at a higher clock
        const int64_t resident = std::min(b, cus * c.slots);
        const double per_cu = resident <= cus ? (double)resident / cus : (double)((resident + cus - 1) / cus);
        const double t = c.t0 + (double)((a + cus - 1) / cus * steps) * c.high +
                         (double)(rounds * steps) * std::max(c.lat, c.mfma * per_cu) +
                         (sp > 1 ? 0.2 + sp * M * K * 8.0 / 8.0 * 1e-6 : 0.0);
        if (t < best_t) {
          best_t = t;
          best = GradPlan{i, (int)full, sp};
        }
      }
    }
  }
  return best;
}

size_t plan_bytes(int64_t M, int64_t K, const GradPlan& p) { return p.splits > 1 ? (size_t)p.splits * M * K * 4 : 0; }

template <int WM, int WN, int FB, int FM, int FN>
hipError_t run(const MxGradArgs& a, const GradPlan& p, float* part, hipStream_t st) {
  constexpr int BN = WN * FN * 32;
  auto k = mx_grad_kernel<WM, WN, FB, FM, FN>;
  const int lds = 2 * stage_bytes(WM * (p.full > 0 ? FB : FM) * 32, BN);
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int kt = (int)((a.N + BK - 1) / BK * a.parts);
  Grid g = {};
  g.tn = (int)((a.K + BN - 1) / BN);
  g.full = p.full;
  g.high = FB > 0 ? (int)((a.M + WM * FB * 32 - 1) / (FB > 0 ? WM * FB * 32 : 1)) : 0;
  g.low = (int)((a.M + WM * FM * 32 - 1) / (WM * FM * 32));
  g.per = (kt + p.splits - 1) / p.splits;
  const int splits = (kt + g.per - 1) / g.per;  // every slice gets at least one stage
  const int64_t wgs = ((int64_t)g.full * g.high + (int64_t)(g.tn - g.full) * g.low) * splits;
  k<<<(unsigned)wgs, WM * WN * 64, lds, st>>>(a.dY, a.W, a.w_scales, a.ep, (int)a.M, (int)a.N, (int)a.L, (int)a.K, (int)a.ld,
                                             a.parts, (int)a.P, g, splits > 1 ? part : nullptr);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  return launch_splitk_reduce(part, splits, a.M, 0, a.K, a.ep, st);
}

}  // namespace

size_t mx_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int parts, const DeviceCaps& caps) {
  return plan_bytes(M, K, pick(M, N, K, parts, caps, true));
}

hipError_t launch_mx_grad(const MxGradArgs& a, const DeviceCaps& caps, void* ws, size_t ws_bytes, hipStream_t st) {
  GradPlan p = pick(a.M, a.N, a.K, a.parts, caps, true);
  if (plan_bytes(a.M, a.K, p) > ws_bytes) p = pick(a.M, a.N, a.K, a.parts, caps, false);
  float* part = static_cast<float*>(ws);
  switch (p.tile) {
    case 0: return run<2, 4, 4, 2, 2>(a, p, part, st);
    case 1: return run<2, 2, 0, 2, 2>(a, p, part, st);
    case 2: return run<1, 4, 0, 2, 1>(a, p, part, st);
    default: return run<1, 4, 0, 1, 1>(a, p, part, st);
  }
}

}  // namespace w4
