// Input gradient of the int8 product (w8a16_mm_t), for gfx950:
//   dX[m][k] = out_rne(sum_n dY[m][n] w[n][k]),  w = rne16(code * scale[n]),
// 16-bit operands, fp32 accumulation.  The contraction runs across the weight's rows, so its
// operand has to be transposed: ds_read_b64_tr_b8 hands each lane eight bytes of one column.
//
// Why w is rounded to dY's type: the scales belong to the contraction, so none of them can wait
// for the sums, and the matrix cores take 16-bit operands; a second product with what the rounding
// leaves over would double the work.  The error is that of a weight stored in that type (8 bits of
// bf16, 11 of fp16).  fp16's short range is not w's: a power of two takes the largest scale of the
// contraction to [2^7, 2^8) (codes to at most 2^15) and the sums are taken back by it, both
// exactly.  Scales 2^21 times smaller than the largest one begin to lose bits.  (Measured: M = 2048,
// (4096, 11008) 187.8 -> 188.4 us, M = 32 17.5 -> 18.2, M = 512, (8192, 2048) 32.4 -> 33.3; that the
// rows' own powers of an fp32 dY were looked for in every launch spilled registers, 188 -> 194, so
// theirs are kernels of their own.)
//
// What bounds it: at M = 2048, (N, K) = (4096, 8192) 118 us, 1165 TFLOP/s, where a bf16 product
// whose weight needs no widening (the library's) takes 111.  The matrix cores are busy 57% of
// the cycles, LDS 38%, and the clock is down to 1.85 GHz; that two waves a SIMD take turns in
// products and in reads behind barriers was slower (126 us), as was each weight widened by two
// waves, with fewer reads of dY (120).
#include <algorithm>
#include <type_traits>

#include "api_common.h"
#include "epilogue.h"
#include "launch.h"
#include "rows.h"

namespace w4 {

namespace {

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

constexpr int BK = 64;  // contraction rows of a stage

// A (FM 32) x (WN 32) tile by WN waves side by side: each wave takes all of the tile's rows and
// 32 columns, so that a weight is widened once in the workgroup.  A stage (64 columns of dY's
// rows, 64 rows of the weight's codes as they are, their 64 scales) goes global -> LDS with
// direct loads, through a ring of three stages.
//   dY rows of 128 bytes: chunk index XOR-ed with (row / 2) % 8; code rows of WN * 32 bytes: with
//   2 (row % 8); both on the source address (no bank conflict counted).
//   v_mfma_f32_32x32x16: lane l supplies dY row l % 32 and weight column l % 32, contraction
//   slots 8 (l / 32) .. + 7 of 16.  The transposing read takes lane l of sixteen to eight bytes
//   of row l / 2 and returns column l of the eight rows.
//   The codes become fp32 products with their scale, rounded once, and 16-bit pairs in registers.
// While product p of a stage's four runs, the operands of p + 1 are read and widened.  The barrier
// in the middle of a stage says that the next one has landed, and that the one before has been
// read, whose slot is then filled; all codes of the next stage are read there, before those
// loads are issued (the compiler waits for every load in flight ahead of a transposing read).
// BACK: row m's sums are multiplied by 2^back[m] as well (F16).
template <int WN, int FM, bool F16, bool BACK>
__device__ __forceinline__ void grad_tile(char* smem, const uint16_t* __restrict__ dY, const int8_t* __restrict__ W,
                                          const float* __restrict__ sw, const Epi& ep, int M, int N, int L, int K, int ld,
                                          int pitch, int m0, int c0, int slice, int per, float* __restrict__ part,
                                          const int* __restrict__ back) {
  constexpr int T = WN * 64, BM = FM * 32, BN = WN * 32, NB = 3;
  constexpr int UA = BM * 8 / T, CB = BN / 16, UB = BK * CB / T;  // chunks a thread loads in a stage
  static_assert(BM * 8 % T == 0 && BK * CB % T == 0, "tile split");
  constexpr int OB = BM * 128, OS = OB + BK * BN, STAGE = OS + BK * 4;  // LDS offsets of codes and scales
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // bytes from the tile's first element to its last row's last one: reads past them return 0
  const uint32_t a_bytes = ((uint32_t)(min(BM, M - m0) - 1) * (uint32_t)ld + (uint32_t)L) * 2u;
  int oa[UA], ca[UA], ob[UB];
#pragma unroll
  for (int i = 0; i < UA; ++i) {
    const int u = tid + i * T, row = u >> 3;
    ca[i] = ((u & 7) ^ ((row >> 1) & 7)) * 8;
    oa[i] = (row * ld + ca[i]) * 2;
  }
#pragma unroll
  for (int i = 0; i < UB; ++i) {
    const int u = tid + i * T, row = u / CB;
    ob[i] = row * pitch + c0 + (((u % CB) ^ (2 * (row & 7) & (CB - 1))) << 4);
  }
  const int k0 = slice * per, KT = min((N + BK - 1) / BK - k0, per);  // this slice's stages
  // loads [lo, hi) of stage kt into ring slot `slot`; past the end the last stage again, never
  // read.  dY's columns past its last one are asked for out of range and so 0.
  constexpr int UL = UA + UB + 1;
  auto dma = [&](int kt, int slot, int lo, int hi) {
    const int n0 = (k0 + min(kt, KT - 1)) * BK;
    const uint32_t rows = (uint32_t)min(BK, N - n0);
    char* base = smem + slot * STAGE;
    const rsrc_t ra = make_rsrc(dY + (size_t)m0 * ld + n0, a_bytes - n0 * 2u);
    const rsrc_t rb = make_rsrc(W + (size_t)n0 * pitch, rows * (uint32_t)pitch);
    const rsrc_t rs = make_rsrc(sw + n0, rows * 4u);
#pragma unroll
    for (int i = 0; i < UL; ++i) {
      if (i < lo || i >= hi) continue;
      if (i < UA)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(base + (i * T + wave * 64) * 16), 16,
                                                 (int)(n0 + ca[i < UA ? i : 0] < L ? oa[i < UA ? i : 0] : 0x7FFFFFFF), 0, 0, 0);
      else if (i < UA + UB)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(base + OB + ((i - UA) * T + wave * 64) * 16), 16,
                                                 (int)ob[i >= UA && i < UA + UB ? i - UA : 0], 0, 0, 0);
      else  // the 64 scales, by every wave (the same bytes), so that all waves count the same loads
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(base + OS), 4, (int)(lane * 4), 0, 0, 0);
    }
  };
  auto sync = [&](auto stages) {
    constexpr int n = decltype(stages)::value * UL;
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((n & 15) | 0xF70 | ((n >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  const int lr = lane & 31, hi = lane >> 5;
  // dY fragment of product p at ^ 32 p; the codes' rows 16 p + 8 hi + (l % 16) / 2
  const int fa = lr * 128 + ((hi ^ ((lr >> 1) & 7)) << 4);
  const int r8 = (lane & 15) >> 1;
  const int fb = OB + (8 * hi + r8) * BN + (((wave * 2 + ((lane >> 4) & 1)) ^ (2 * r8 & (CB - 1))) << 4) + 8 * (lane & 1);
  u32x4 x[2][FM], y[2];
  i32x2 raw[4], coming[4];
  f32x4 sc[2][2];
  auto read_x = [&](const char* base, int p, u32x4 (&v)[FM]) {
#pragma unroll
    for (int i = 0; i < FM; ++i) v[i] = *reinterpret_cast<const u32x4*>(base + (fa ^ (32 * p)) + i * 32 * 128);
  };
  auto read_raw = [&](char* base, i32x2 (&v)[4]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(base + fb + p * 16 * BN));
  };
  auto read_sc = [&](const char* base, int p, f32x4 (&s)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h] = *reinterpret_cast<const f32x4*>(base + OS + (16 * p + 8 * hi + 4 * h) * 4);
  };
  // fp16: the power of two that takes the largest finite scale of this slice to [2^7, 2^8)
  int power = 0;
  float up = 1.0f;
  auto widen = [&](const i32x2& v, const f32x4 (&s)[2], u32x4& o) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) f[b] = (float)(int8_t)(v[h] >> (8 * b)) * (F16 ? s[h][b] * up : s[h][b]);
      o[2 * h] = F16 ? pack_f16x2(f[0], f[1]) : pack_bf16x2(f[0], f[1]);
      o[2 * h + 1] = F16 ? pack_f16x2(f[2], f[3]) : pack_bf16x2(f[2], f[3]);
    }
  };
  f32x16 acc[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;

  // fp16: the largest finite scale.  A thread's first eight are asked for ahead of the stages (loads
  // return in order), the others behind them.
  const int n_end = min(N, (k0 + KT) * BK);
  uint32_t peak = 0;
  auto take = [&](uint32_t u) { peak = umax(peak, (u & 0x7FFFFFFFu) < 0x7F800000u ? u & 0x7FFFFFFFu : 0u); };
  auto scales8 = [&](int n) {
    if (n + 8 <= n_end) return load_raw8<W4_DT_F32>(sw + n);
    return n < n_end ? load_raw8_part<W4_DT_F32>(sw + n, n_end - n, 0u) : Raw8<W4_DT_F32>{};
  };
  Raw8<W4_DT_F32> first;
  if constexpr (F16) {
    first = scales8(k0 * BK + tid * 8);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int k = 0; k < NB - 1; ++k) dma(k, k, 0, UL);
  if constexpr (F16) {
    __shared__ uint32_t peaks[WN];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 8; ++j) take(first.q[j >> 2][j & 3]);
#pragma unroll 4
    for (int n = k0 * BK + (tid + T) * 8; n < n_end; n += T * 8) {
      const Raw8<W4_DT_F32> s8 = scales8(n);
#pragma unroll
      for (int j = 0; j < 8; ++j) take(s8.q[j >> 2][j & 3]);
    }
    peak = wave_umax(peak);
    if (lane == 0) peaks[wave] = peak;
    // this wave's LDS write done, then a barrier with no fence, which would wait for the stages
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < WN; ++i) peak = umax(peak, peaks[i]);
    if (peak != 0) power = min(134 - (int)(__builtin_amdgcn_readfirstlane(peak) >> 23), 126);
    up = __uint_as_float((uint32_t)(127 + power) << 23);
  }
  sync(std::integral_constant<int, NB - 2>());
  read_x(smem, 0, x[0]);
  read_raw(smem, raw);
  read_sc(smem, 0, sc[0]);
  read_sc(smem, 1, sc[1]);
  widen(raw[0], sc[0], y[0]);
  int slot = 0;
  for (int kt = 0; kt < KT; ++kt) {
    const int next = slot == NB - 1 ? 0 : slot + 1, spare = slot == 0 ? NB - 1 : slot - 1;
    char* now_b = smem + slot * STAGE;
    char* next_b = smem + next * STAGE;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int cur = p & 1, nxt = cur ^ 1;
      if (p == 2) {
        sync(std::integral_constant<int, NB - 3>());
        read_raw(next_b, coming);
      }
      __builtin_amdgcn_sched_barrier(0);
      read_x(p < 3 ? now_b : next_b, (p + 1) & 3, x[nxt]);
      widen(p < 3 ? raw[p + 1] : coming[0], sc[nxt], y[nxt]);
      read_sc(p < 2 ? now_b : next_b, (p + 2) & 3, sc[cur]);
#pragma unroll
      for (int i = 0; i < FM; ++i) acc[i] = mfma_op<F16>(x[cur][i], y[cur], acc[i]);
      if (p >= 2) dma(kt + NB - 1, spare, p == 2 ? 0 : UL / 2, p == 2 ? UL / 2 : UL);
      // issue: a product, then a little of everything else
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                     // product
        __builtin_amdgcn_sched_group_barrier(0x100, (FM + 1 + FM) / FM, 0);    // LDS reads
        __builtin_amdgcn_sched_group_barrier(0x002, ((F16 ? 27 : 19) + FM) / FM, 0);  // widening
        if (p >= 2) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);         // direct loads
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) raw[p] = coming[p];
    slot = next;
  }
  // no direct LDS load may land after the workgroup's LDS is handed on
  __builtin_amdgcn_s_waitcnt(0x0070);
  const int cbase = c0 + wave * 32, mbase = m0 + hi * 4, c = cbase + lr;
  if constexpr (BACK) {
    // by the weight's power and the row's own in one step: the product of the two may be no fp32
    const rsrc_t rb = make_rsrc(back, (uint32_t)M * 4u);  // M < 2^30
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      __builtin_amdgcn_sched_barrier(0);  // sixteen rows' at a time: all at once would spill
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const u32x4 b = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                      rb, (int)((uint32_t)(mbase + i * 32 + g * 8) * 4u), 0, 0));
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][g * 4 + q] = __builtin_ldexpf(acc[i][g * 4 + q], (int)b[q] - power);
      }
    }
  } else if constexpr (F16) {
    const float down = __uint_as_float((uint32_t)(127 - power) << 23);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][r] *= down;
  }
  if (part == nullptr && epi_wide(ep, K) != 0) {
    const EpiQuad q = epi_quad(ep, cbase + (lr & ~3), K);
#pragma unroll
    for (int i = 0; i < FM; ++i) epi_put_block_wide(q, acc[i], mbase + i * 32, M, lane);
    return;
  }
  if (c >= K) return;
  if (part != nullptr) {  // a slice's sums go to its own [M][K] plane
    float* out = part + (size_t)slice * M * K + c;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = mbase + i * 32 + (r >> 2) * 8 + (r & 3);
        if (m < M) out[(size_t)m * K] = acc[i][r];
      }
    return;
  }
  const EpiCol col = epi_col(ep, c);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int m = mbase + i * 32 + (r >> 2) * 8 + (r & 3);
      if (m < M) epi_put(ep, col, m, acc[i][r]);
    }
}

// Work of a launch: the first `full` column tiles in (FB 32)-row tiles, the columns left in
// (FM 32)-row tiles; all of that once for each slice of the contraction.
struct Grid {
  int full, tn;   // column tiles of the first kind, and in all
  int high, low;  // row tiles of the two kinds
  int per;        // stages of a slice
};

template <int WN, int FB, int FM, bool F16, bool BACK>
__global__ __launch_bounds__(WN * 64) void w8_grad_kernel(const uint16_t* __restrict__ dY, const int8_t* __restrict__ W,
                                                          const float* __restrict__ sw, const Epi ep, int M, int N, int L,
                                                          int K, int ld, int pitch, const Grid g, float* __restrict__ part,
                                                          const int* __restrict__ back) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int n_high = FB > 0 ? g.full * g.high : 0, n_all = n_high + (g.tn - g.full) * g.low;
  const int slice = blockIdx.x / (unsigned)n_all;
  int at = blockIdx.x - (unsigned)slice * n_all;
  const bool high = at < n_high;
  if (!high) at -= n_high;
  // Order: groups of eight tile rows, tile columns, rows of the group.  Workgroups go to the eight
  // XCDs in turn, so an XCD's 256-row tiles share a tile row (2% better than the order below);
  // of the smaller tiles, which the L2 feeds, each XCD gets a contiguous part.
  const int rows = high ? g.high : g.low, cols = high ? g.full : g.tn - g.full;
  const int per_xcd = (n_all - n_high) >> 3, left = (n_all - n_high) & 7, xcd = at & 7;
  const int tile = high ? at : xcd * per_xcd + min(xcd, left) + (at >> 3);
  const int grp = tile / (8 * cols), in_grp = tile - grp * 8 * cols, rows_grp = min(8, rows - grp * 8);
  const int tr = grp * 8 + in_grp % rows_grp, tc = in_grp / rows_grp + (high ? 0 : g.full);
  if constexpr (FB > 0)
    if (high) {
      grad_tile<WN, FB, F16, BACK>(smem, dY, W, sw, ep, M, N, L, K, ld, pitch, tr * FB * 32, tc * WN * 32, slice, g.per, part,
                              back);
      return;
    }
  grad_tile<WN, FM, F16, BACK>(smem, dY, W, sw, ep, M, N, L, K, ld, pitch, tr * FM * 32, tc * WN * 32, slice, g.per, part, back);
}

// Tiles of WN * 32 columns: FB * 32 rows (0: none) and FM * 32 rows, and what one stage of them
// takes, in us on MI355X (fitted to some 20 sizes, M = 8 to 5000): high, of an FB tile; lat, the
// least time of a stage of an FM tile; mfma, a workgroup's share of the CU's matrix cores; and t0,
// a launch's start, first loads and stores.
struct Tile {
  int wn, fb, fm, slots;  // slots: workgroups that a CU's LDS holds
  double t0, high, lat, mfma;
};
constexpr Tile kTiles[] = {
    {8, 8, 4, 1, 9.0, 1.70, 0.78, 0.95},
    {4, 0, 4, 2, 6.0, 0.00, 0.56, 0.50},
    {4, 0, 2, 3, 5.0, 0.00, 0.48, 0.32},
    {4, 0, 1, 4, 5.0, 0.00, 0.46, 0.28},
};

struct GradPlan {
  int tile = 0, full = 0, splits = 1;
};

// The plan with the least estimated time: rounds of workgroups, each the contraction's stages; a
// split adds a launch (3 us) and the write and read of its planes (8 TB/s: they fit the
// caches).  256-row tiles take none of the columns, all, or those that make whole rounds, the
// last, partial round then being one of 128-row tiles: at M = 2048, (N, K) = (4096, 11008)
// 196 us with 256-row tiles alone, 190 with 128-row tiles, 172 with both.
GradPlan pick(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps, bool allow_split) {
  const int64_t cus = caps.cus > 0 ? caps.cus : 256, kt = (N + BK - 1) / BK;
  GradPlan best;
  double best_t = 1e30;
  for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
    const Tile& c = kTiles[i];
    const int64_t tn = (K + c.wn * 32 - 1) / (c.wn * 32), low = (M + c.fm * 32 - 1) / (c.fm * 32);
    const int64_t high = c.fb > 0 ? (M + c.fb * 32 - 1) / (c.fb * 32) : 0;
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
                         (sp > 1 ? 3.0 + sp * M * K * 8.0 / 8.0 * 1e-6 : 0.0);
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

template <int WN, int FB, int FM>
hipError_t run(const W8GradArgs& a, const GradPlan& p, float* part, hipStream_t st) {
  auto k = !a.f16 ? w8_grad_kernel<WN, FB, FM, false, false>
           : a.back == nullptr ? w8_grad_kernel<WN, FB, FM, true, false>
                               : w8_grad_kernel<WN, FB, FM, true, true>;
  constexpr int rows = (FB > FM ? FB : FM) * 32;
  const int lds = 3 * ((p.full > 0 ? rows : FM * 32) * 128 + BK * WN * 32 + BK * 4);
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int kt = (int)((a.N + BK - 1) / BK);
  Grid g = {};
  g.tn = (int)((a.K + WN * 32 - 1) / (WN * 32));
  g.full = p.full;
  g.high = FB > 0 ? (int)((a.M + FB * 32 - 1) / (FB > 0 ? FB * 32 : 1)) : 0;
  g.low = (int)((a.M + FM * 32 - 1) / (FM * 32));
  g.per = (kt + p.splits - 1) / p.splits;
  const int splits = (kt + g.per - 1) / g.per;  // every slice gets at least one stage
  const int64_t wgs = ((int64_t)g.full * g.high + (int64_t)(g.tn - g.full) * g.low) * splits;
  k<<<(unsigned)wgs, WN * 64, lds, st>>>(a.dY, a.W, a.w_scales, a.ep, (int)a.M, (int)a.N, (int)a.L, (int)a.K, (int)a.ld,
                                         (int)a.pitch, g, splits > 1 ? part : nullptr, a.back);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  return launch_splitk_reduce(part, splits, a.M, 0, a.K, a.ep, st);
}

// dY rows copied to an aligned pitch, zeros past column N.
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

size_t w8_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps) {
  return plan_bytes(M, K, pick(M, N, K, caps, true));
}

hipError_t launch_w8_grad(const W8GradArgs& a, const DeviceCaps& caps, void* ws, size_t ws_bytes, hipStream_t st) {
  GradPlan p = pick(a.M, a.N, a.K, caps, true);
  if (plan_bytes(a.M, a.K, p) > ws_bytes) p = pick(a.M, a.N, a.K, caps, false);
  float* part = static_cast<float*>(ws);
  switch (p.tile) {
    case 0: return run<8, 8, 4>(a, p, part, st);
    case 1: return run<4, 0, 4>(a, p, part, st);
    case 2: return run<4, 0, 2>(a, p, part, st);
    default: return run<4, 0, 1>(a, p, part, st);
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
