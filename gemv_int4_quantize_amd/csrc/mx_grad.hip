// Input gradient of the microscaled 4-bit product (mx4_mm_t), for gfx950:
//   dX[m][k] = out_rne(sum_n dY[m][n] w[n][k]),  w = code * 2^(exponent - 127),
// fp32 accumulation.  The contraction runs across the weight's rows, along which the exponents
// change with every row, so the 4-bit matrix instructions do not apply; but w has two significant
// bits, so bf16 holds it exactly, and dY enters as bf16 parts whose sum it is (one of bf16, two of
// fp16, three of fp32): the parts lengthen the contraction, and nothing is rounded before the sums.
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

// One workgroup of WM x WN waves computes a (WM FM 32) x (WN FN 32) tile.  A stage is 64 columns of
// dY's rows and 64 rows of the weight.
//   dY goes global -> LDS with direct loads through a ring of NB slots, rows of 128 bytes, their
//   16-byte chunk index XOR-ed with (row / 2) % 8 on the source address.
//   A thread takes blocks of 32 weight columns (16 bytes and their exponent) through registers: read
//   one stage ahead, widened once in the workgroup and written to LDS as 64 bytes of bf16, in one of
//   two slots.  A row's 64-byte pieces are at piece ^ (row % 4), and a piece's 16-byte quarters at
//   quarter ^ (piece / 4 % 2 + 2 (row % 2)): sixteen lanes' writes, and the 4-row reads of half a
//   wave, hit distinct banks.
//   v_mfma_f32_32x32x16_bf16: lane l supplies dY row l % 32 and weight column l % 32, contraction
//   slots 8 (l / 32) .. + 7 of 16.  A transposing read takes sixteen lanes to 4 rows of 16 columns
//   and returns lane l column l of the four rows; two make an operand.
// A stage's transposed operands are all read at its start, ahead of the direct loads (the compiler
// waits for every load in flight ahead of a transposing read).
template <int WM, int WN, int FM, int FN, int NB>
__device__ __forceinline__ void grad_tile(char* smem, const uint16_t* __restrict__ dY, const uint8_t* __restrict__ W,
                                          const uint8_t* __restrict__ we, const Epi& ep, int M, int N, int L, int K, int ld,
                                          int parts, int P, int m0, int c0, int slice, int per, float* __restrict__ part) {
  constexpr int T = WM * WN * 64, BM = WM * FM * 32, BN = WN * FN * 32;
  constexpr int CB = BN / 32, UA = BM * 8 / T, UB = BK * CB / T;  // chunks a thread loads in a stage
  static_assert(BM * 8 % T == 0 && BK * CB % T == 0 && (CB & (CB - 1)) == 0 && CB >= 4, "tile split");
  constexpr int SA = BM * 128, SW = BK * BN * 2, OW = NB * SA;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int row = P >> 1, erow = P >> 5;
  const int nst = (N + BK - 1) / BK;  // stages of a part
  const int k0 = slice * per, KT = min(nst * parts - k0, per);
  int oa[UA], ca[UA], ob[UB], oe[UB];
#pragma unroll
  for (int i = 0; i < UA; ++i) {
    const int u = tid + i * T, r = u >> 3;
    ca[i] = ((u & 7) ^ ((r >> 1) & 7)) * 8;
    oa[i] = (r * parts * ld + ca[i]) * 2;
  }
  int at_w[UB];
#pragma unroll
  for (int i = 0; i < UB; ++i) {
    const int u = tid + i * T, r = u / CB, c = u % CB;
    ob[i] = r * row + (c0 >> 1) + c * 16;
    oe[i] = r * erow + (c0 >> 5) + c;
    at_w[i] = OW + r * (BN * 2) + ((c ^ (r & 3)) << 6) + ((((c >> 2) & 1) | (r & 1) << 1) << 4);
  }
  // stage kt (past the end the last one again, never used): its part and its first row
  auto stage = [&](int kt, int* pt) {
    const int s = k0 + min(kt, KT - 1);
    *pt = s / nst;
    return (s - *pt * nst) * BK;
  };
  const uint32_t a_bytes = (uint32_t)min(BM, M - m0) * (uint32_t)(parts * ld) * 2u;
  auto dma = [&](int kt, int slot) {
    int pt;
    const int n0 = stage(kt, &pt);
    const uint32_t skip = (uint32_t)(pt * ld + n0);
    // columns past the last one are asked for out of range and so 0
    const rsrc_t ra = mx_rsrc(dY + (size_t)m0 * parts * ld + skip, a_bytes - skip * 2u);
    char* base = smem + slot * SA + wave * 1024;
#pragma unroll
    for (int i = 0; i < UA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(base + i * T * 16), 16,
                                               (int)(n0 + ca[i] < L ? oa[i] : 0x7FFFFFFF), 0, 0, 0);
  };
  u32x4 wr[UB];
  uint32_t er[UB];
  auto load_w = [&](int kt) {
    int pt;
    const int n0 = stage(kt, &pt);
    const uint32_t rows = (uint32_t)min(BK, N - n0);
    const rsrc_t rb = mx_rsrc(W + (size_t)n0 * row, rows * (uint32_t)row);
    const rsrc_t re = mx_rsrc(we + (size_t)n0 * erow, rows * (uint32_t)erow);
#pragma unroll
    for (int i = 0; i < UB; ++i) {
      wr[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rb, ob[i], 0, 0));
      er[i] = __builtin_amdgcn_raw_buffer_load_b8(re, oe[i], 0, 0);
    }
  };
  auto widen = [&](int slot) {
#pragma unroll
    for (int i = 0; i < UB; ++i) {
      const float p = mx_power(er[i]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<u32x4*>(smem + ((at_w[i] + slot * SW) ^ (q << 4))) = mx_bf16x8(wr[i][q], p);
    }
  };
  // all but the last NB - 2 stages of dY landed, this wave's LDS reads and writes done, then a
  // barrier with no fence (a fence would wait for every load in flight)
  auto sync = [&]() {
    constexpr int n = 2 * UB + (NB - 2) * (UA + 2 * UB);
    static_assert(n < 64, "the wait's counter");
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((n & 15) | 0x70 | ((n >> 4) << 14));
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
  u32x4 x[2][FM];
  u32x2 b[4][FN][2];
  auto read_x = [&](const char* base, int p, u32x4 (&v)[FM]) {
#pragma unroll
    for (int i = 0; i < FM; ++i) v[i] = *reinterpret_cast<const u32x4*>(base + (fa ^ (32 * p)) + i * 32 * 128);
  };

  load_w(0);
#pragma unroll
  for (int k = 0; k < NB - 1; ++k) dma(k, k);
  widen(0);
  load_w(1);
  int slot = 0;
  for (int kt = 0; kt < KT; ++kt) {
    sync();
    char* wb = smem + (kt & 1) * SW;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          b[p][j][h] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                     (lds_s16x4*)(wb + fb[j] + (16 * p + 4 * h) * (BN * 2))));
    const char* base = smem + slot * SA;
    read_x(base, 0, x[0]);
    __builtin_amdgcn_sched_barrier(0);
    dma(kt + NB - 1, slot == 0 ? NB - 1 : slot - 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if (p < 3) read_x(base, p + 1, x[(p + 1) & 1]);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = mfma_op<false>(x[p & 1][i], u32x4{b[p][j][0][0], b[p][j][0][1], b[p][j][1][0], b[p][j][1][1]}, acc[i][j]);
      if (p == 1) widen((kt + 1) & 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    load_w(kt + 2);
    slot = slot == NB - 1 ? 0 : slot + 1;
  }
  // no direct LDS load may land after the workgroup's LDS is handed on
  __builtin_amdgcn_s_waitcnt(0x0070);
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

// Tiles of one kind (tm x tn), all of them once for each slice.  Workgroups go to the eight XCDs in
// turn; each XCD gets a contiguous part of the work, in the order: slices, groups of eight tile
// rows, tile columns, rows of the group.
template <int WM, int WN, int FM, int FN, int NB>
__global__ __launch_bounds__(WM * WN * 64) void mx_grad_kernel(const uint16_t* __restrict__ dY, const uint8_t* __restrict__ W,
                                                               const uint8_t* __restrict__ we, const Epi ep, int M, int N, int L,
                                                               int K, int ld, int parts, int P, int tm, int tn, int per,
                                                               float* __restrict__ part) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int per_xcd = gridDim.x >> 3, left = gridDim.x & 7, xcd = blockIdx.x & 7;
  const int work = xcd * per_xcd + min(xcd, left) + (blockIdx.x >> 3);
  const int slice = work / (tm * tn), tile = work - slice * tm * tn;
  const int grp = tile / (8 * tn), in_grp = tile - grp * 8 * tn, rows_grp = min(8, tm - grp * 8);
  const int ti = grp * 8 + in_grp % rows_grp, tj = in_grp / rows_grp;
  grad_tile<WM, WN, FM, FN, NB>(smem, dY, W, we, ep, M, N, L, K, ld, parts, P, ti * WM * FM * 32, tj * WN * FN * 32, slice, per,
                                part);
}

// Tiles, and what one stage of them takes, in us on MI355X: lat, the least time of a stage; mfma, a
// workgroup's share of the CU's matrix cores; and t0, a launch's start, first loads and stores.
struct Tile {
  int bm, bn, slots;  // slots: workgroups that a CU's LDS holds
  double t0, lat, mfma;
};
constexpr Tile kTiles[] = {
    {256, 256, 1, 9.0, 1.30, 1.60},
    {128, 128, 2, 6.0, 0.56, 0.50},
    {64, 128, 2, 5.0, 0.48, 0.32},
    {32, 128, 2, 5.0, 0.46, 0.28},
};

struct GradPlan {
  int tile = 0, splits = 1;
};

// The plan with the least estimated time: rounds of workgroups, each the contraction's stages; a
// split adds a launch and the write and read of its planes.
GradPlan pick(int64_t M, int64_t N, int64_t K, int parts, const DeviceCaps& caps, bool allow_split) {
  const int64_t cus = caps.cus > 0 ? caps.cus : 256, kt = (N + BK - 1) / BK * parts;
  GradPlan best;
  double best_t = 1e30;
  for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
    const Tile& c = kTiles[i];
    const int64_t tn = (K + c.bn - 1) / c.bn, tm = (M + c.bm - 1) / c.bm;
    for (int sp = 1; sp <= (allow_split ? 8 : 1); sp *= 2) {
      if (sp > 1 && kt / sp < 4) break;
      const int64_t steps = (kt + sp - 1) / sp;
      const int64_t wgs = tm * tn * sp, rounds = (wgs + cus * c.slots - 1) / (cus * c.slots);
      // workgroups of the fullest CU
      const int64_t resident = std::min(wgs, cus * c.slots);
      const double per_cu = resident <= cus ? (double)resident / cus : (double)((resident + cus - 1) / cus);
      const double t = c.t0 + (double)(rounds * steps) * std::max(c.lat, c.mfma * per_cu) +
                       (sp > 1 ? 3.0 + sp * M * K * 8.0 / 8.0 * 1e-6 : 0.0);
      if (t < best_t) {
        best_t = t;
        best = GradPlan{i, sp};
      }
    }
  }
  return best;
}

size_t plan_bytes(int64_t M, int64_t K, const GradPlan& p) { return p.splits > 1 ? (size_t)p.splits * M * K * 4 : 0; }

template <int WM, int WN, int FM, int FN, int NB>
hipError_t run(const MxGradArgs& a, const GradPlan& p, float* part, hipStream_t st) {
  constexpr int BM = WM * FM * 32, BN = WN * FN * 32;
  constexpr int lds = NB * BM * 128 + 2 * BK * BN * 2;
  auto k = mx_grad_kernel<WM, WN, FM, FN, NB>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int kt = (int)((a.N + BK - 1) / BK * a.parts);
  const int tm = (int)((a.M + BM - 1) / BM), tn = (int)((a.K + BN - 1) / BN);
  const int per = (kt + p.splits - 1) / p.splits;
  const int splits = (kt + per - 1) / per;  // every slice gets at least one stage
  k<<<(unsigned)((int64_t)tm * tn * splits), WM * WN * 64, lds, st>>>(a.dY, a.W, a.w_scales, a.ep, (int)a.M, (int)a.N, (int)a.L,
                                                                     (int)a.K, (int)a.ld, a.parts, (int)a.P, tm, tn, per,
                                                                     splits > 1 ? part : nullptr);
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
    case 1: return run<2, 2, 2, 2, 2>(a, p, part, st);
    case 2: return run<1, 4, 2, 1, 2>(a, p, part, st);
    default: return run<1, 4, 1, 1, 2>(a, p, part, st);
  }
}

}  // namespace w4
