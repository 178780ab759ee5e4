// Products of microscaled 4-bit rows for few tokens, for gfx950: one to eight that are quantized by the same
// launch (decode), or up to 32 whose codes are ready.  The weight is read once, and its bytes set the time.
//
// A workgroup stays for several groups of 16 RT channels, its tokens' codes in LDS; its waves share out
// the contraction in 256-column units.  A wave has its own ring of units in LDS, filled by direct loads,
// and its next units, of this group or the one after it, are on their way while the sums of a group are put
// together.  (Loads into registers, each lane at a row of its own, cost the vector caches a tag for every 16
// bytes: one token at (N, K) = (12288, 4096) 12.9 us, 7.0 here.)  In a captured graph, one token:
// (2048, 2048) 3.2 us, (4096, 11008) 6.6, (16384, 16384) 30.8 (4.6 TB/s).
// v_mfma_scale_f32_16x16x128_f8f6f4 with channels as rows and tokens as columns: lane l supplies a
// block of 32 columns of channel l % 16 and of token l % 16, the same columns of both, and their two
// exponents, and holds token l % 16 of channels 4 (l / 16) .. + 3.
#include <algorithm>

#include "api_common.h"
#include "epilogue.h"
#include "launch.h"
#include "mx.h"

namespace w4 {

namespace {

constexpr int kNonTemporal = 2;       // cache-policy operand of a load
constexpr int kMaxM = 8;              // tokens
// Columns of all tokens, up to four of them and up to eight.  Every workgroup quantizes them, and past these
// a launch that quantizes once and one for ready codes are as fast.  (N, K) = (12288, 4096): 8 tokens 9.7 us
// here, 9.8 so, 10 tokens 11.6, 10.2; (4096, 11008): 4 tokens 8.3, 8.7, 6 tokens 13.1, 8.9; (8192, 2048):
// 8 tokens 5.5, 6.3, 10 tokens 6.9, 6.5; (16384, 16384): 2 tokens 33, 3 tokens 37.5, 32.9.
constexpr int64_t max_columns(int64_t M) { return M <= 4 ? 45056 : 32768; }
constexpr int kFewM = 32;   // tokens whose codes are ready
constexpr int kReadyM = 2;  // of them, in the decode kernel

// The tokens in LDS: exponents [M][P / 32 rounded up to 8] (a unit's eight are read as one), then codes
// [M][P / 2 + 16] (the pad keeps the tokens' rows in distinct banks).
constexpr int exponents_pitch(int64_t P) { return (int)(((P >> 5) + 7) & ~(int64_t)7); }
constexpr int codes_at(int64_t M, int64_t P) { return (int)((M * exponents_pitch(P) + 15) & ~(int64_t)15); }
constexpr int64_t token_lds(int64_t M, int64_t P) { return codes_at(M, P) + M * ((P >> 1) + 16); }

// A unit in LDS: 128 bytes a row, the 16-byte chunks (a block of 32 columns each) at chunk ^ (row / 2 % 8),
// on the source address, so that reads of 16 rows hit distinct banks; then 8 exponents a row, of 32 rows.
constexpr int slot_bytes(int RT) { return RT * 2048 + 256; }

// MT: tokens that there is room for.  XDT: -1: their codes from memory; else the dtype of float tokens.
// Loads return in order, so the tokens are asked for before the weights: C chunks of eight per thread
// (what is left of more or longer tokens is read behind them).
template <int NW, int RT, int SLOTS, int MT, int XDT, int C>
__global__ __launch_bounds__(NW * 64) void mx_decode_kernel(const uint8_t* __restrict__ W, const uint8_t* __restrict__ we,
                                                            const uint8_t* __restrict__ A, const uint8_t* __restrict__ ae,
                                                            const void* __restrict__ X, int64_t ldx, int M, int N, int K,
                                                            int P, const Epi ep) {
  constexpr int T = NW * 64, nD = 2 * RT + 1;  // loads of a unit
  constexpr int SLOT = slot_bytes(RT);
  extern __shared__ __attribute__((aligned(16))) char smem[];  // rings [NW][SLOTS][SLOT], then the tokens
  __shared__ float sums[2][NW][RT * 16][MT + 1];               // of groups in turn
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int units = (P + 255) >> 8, groups = (N + RT * 16 - 1) / (RT * 16);
  const int row = P >> 1, erow = P >> 5;  // bytes of a row's codes and exponents
  const int r16 = lane & 15, q4 = lane >> 4;
  char* own = smem + wave * (SLOTS * SLOT);
  char* tokens = smem + NW * SLOTS * SLOT;
  const int at_codes = codes_at(M, P), epitch = exponents_pitch(P);

  int off[2];  // where a lane's loads of 8 rows begin
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = 8 * j + (lane >> 3);
    off[j] = r * row + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
  }
  const int eoff = (lane >> 1) * erow + (lane & 1) * 4;
  // A group of channels and the unit (one step also where the wave has none).
  struct Place {
    int group, u;
  };
  auto advance = [&](Place& p) {
    p.u += NW;
    if (p.u < units) return;
    p.u = wave;
    p.group += gridDim.x;
  };
  // channels past the last one, and all of a place past the end: 0, without a request
  auto load = [&](const Place& p, int slot) {
    char* at = own + slot * SLOT;
    const size_t n0 = (size_t)p.group * (RT * 16);
    const int rows = p.group < groups && p.u < units ? min(RT * 16, N - (int)n0) : 0;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const rsrc_t rw = mx_rsrc(W + (n0 + r * 16) * row, __builtin_amdgcn_readfirstlane(max(0, rows - r * 16) * (uint32_t)row));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(at + r * 2048 + j * 1024), 16, (int)off[j], (int)(p.u * 128), 0,
                                                 kNonTemporal);
    }
    const rsrc_t re = mx_rsrc(we + n0 * erow, __builtin_amdgcn_readfirstlane(rows * (uint32_t)erow));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(re, (lds_void*)(at + RT * 2048), 4, (int)eoff, (int)(p.u * 8), 0, 0);
  };
  Place now = {(int)blockIdx.x, wave}, ahead = now;
  auto first_loads = [&]() {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < SLOTS - 1; ++k) {
      load(ahead, k);
      advance(ahead);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  if constexpr (XDT >= 0) {
    typedef typename Elem<XDT>::type E;
    const int ch = P >> 3;
    auto chunk = [&](int m, int c) {
      const E* p = static_cast<const E*>(X) + m * ldx + c * 8;
      if (c * 8 + 8 <= K) return load_raw8<XDT>(p);
      return c * 8 < K ? load_raw8_part<XDT>(p, K - c * 8, 0u) : Raw8<XDT>{};
    };
    auto put = [&](int m, int c, bool in, const Raw8<XDT>& r) {
      uint32_t e;
      const uint32_t code = mx_chunk<XDT>(r, &e);
      if (in) {
        *reinterpret_cast<uint32_t*>(tokens + at_codes + m * (row + 16) + c * 4) = code;
        if ((c & 3) == 0) tokens[m * epitch + (c >> 2)] = (char)e;
      }
    };
    if constexpr (MT == 4) {  // the same chunks of each token
      constexpr int CT = C / 4;
      Raw8<XDT> held[MT][CT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          held[m][c] = Raw8<XDT>{};
          if (m < M && tid + c * T < ch) held[m][c] = chunk(m, tid + c * T);
        }
      first_loads();
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m >= M) break;
#pragma unroll
        for (int c = 0; c < CT; ++c) put(m, tid + c * T, tid + c * T < ch, held[m][c]);
        for (int c = tid + CT * T; c - tid < ch; c += T) put(m, c, c < ch, c < ch ? chunk(m, c) : Raw8<XDT>{});
      }
    } else {  // the chunks of all tokens in a row
      const uint32_t all = (uint32_t)(M * ch);
      Raw8<XDT> held[C];
      auto fetch = [&](uint32_t i0) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t i = i0 + tid + c * T;
          held[c] = i < all ? chunk((int)(i / ch), (int)(i % ch)) : Raw8<XDT>{};
        }
      };
      fetch(0);
      first_loads();
      for (uint32_t i0 = 0; i0 < all; i0 += C * T) {
        if (i0 > 0) fetch(i0);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t i = i0 + tid + c * T;
          put((int)(i / ch), (int)(i % ch), i < all, held[c]);
        }
      }
    }
  } else {
    for (int m = 0; m < M; ++m) {
      for (int c = tid; c < row / 16; c += T)
        *reinterpret_cast<u32x4*>(tokens + at_codes + m * (row + 16) + c * 16) =
            *reinterpret_cast<const u32x4*>(A + (size_t)m * row + c * 16);
      for (int c = tid; c < erow / 4; c += T)
        *reinterpret_cast<uint32_t*>(tokens + m * epitch + c * 4) = *reinterpret_cast<const uint32_t*>(ae + (size_t)m * erow + c * 4);
    }
    first_loads();
  }
  // this wave's LDS reads and writes done, then a barrier with no fence, which would wait for the weights
  auto barrier = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  barrier();

  f32x4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int m0 = min(r16, M - 1);
  const char* xc = tokens + at_codes + m0 * (row + 16) + q4 * 16;
  const char* xe = tokens + m0 * epitch;
  int slot = 0, turn = 0;
  while (now.group < groups) {
    load(ahead, slot == 0 ? SLOTS - 1 : slot - 1);
    advance(ahead);
    {
      constexpr int n = (SLOTS - 1) * nD;
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt((n & 15) | 0xF70 | ((n >> 4) << 14));
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    }
    if (now.u < units) {
      const char* at = own + slot * SLOT;
      const u32x2 ex = *reinterpret_cast<const u32x2*>(xe + now.u * 8);
      u32x2 ew[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) ew[r] = *reinterpret_cast<const u32x2*>(at + RT * 2048 + (r * 16 + r16) * 8);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && now.u * 256 + 128 >= P) break;  // the row ends in the middle of its last unit
        const u32x4 x = *reinterpret_cast<const u32x4*>(xc + now.u * 128 + h * 64);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const u32x4 w = *reinterpret_cast<const u32x4*>(at + r * 2048 + r16 * 128 + (((4 * h + q4) ^ (r16 >> 1)) << 4));
          acc[r] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(w), mx_operand(x), acc[r], kFp4, kFp4, 0,
                                                                    (int)(ew[r][h] >> (8 * q4)), 0, (int)(ex[h] >> (8 * q4)));
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    slot = slot == SLOTS - 1 ? 0 : slot + 1;
    if (now.u + NW >= units) {
      // the group's sums, by waves in turn.  One barrier a group: the next one's sums have a place of their
      // own, and when they are written every wave has passed this one's.
      float(*sum)[RT * 16][MT + 1] = sums[turn & 1];
      if (r16 < M) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[wave][r * 16 + q4 * 4 + i][r16] = acc[r][i];
      }
      barrier();
      for (int i = ((wave + turn) & (NW - 1)) * 64 + lane; i < M * (RT * 16); i += T) {
        const int m = i / (RT * 16), c = i % (RT * 16), n = now.group * (RT * 16) + c;
        if (n >= N) continue;
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NW; ++v) s += sum[v][c][m];
        epi_put(ep, epi_col(ep, n), m, s);
      }
      ++turn;
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    advance(now);
  }
  __builtin_amdgcn_s_waitcnt(0x0070);  // no direct LDS load may land after the workgroup's LDS is handed on
}

template <int NW, int RT, int SLOTS, int MT, int XDT, int C>
hipError_t run(const MxArgs& a, const DeviceCaps& caps, hipStream_t st) {
  static_assert((NW & (NW - 1)) == 0, "waves in turn");
  const int64_t lds = NW * SLOTS * slot_bytes(RT) + token_lds(a.M, a.P);
  constexpr int64_t fixed = 2 * NW * RT * 16 * (MT + 1) * 4;
  auto k = mx_decode_kernel<NW, RT, SLOTS, MT, XDT, C>;
  if (lds + fixed > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  const int64_t groups = (a.N + RT * 16 - 1) / (RT * 16), per_cu = std::max<int64_t>(1, 160 * 1024 / (lds + fixed));
  k<<<(unsigned)std::min<int64_t>(groups, per_cu * caps.cus), NW * 64, lds, st>>>(a.W, a.w_scales, a.A, a.a_scales, a.X, a.ldx,
                                                                                (int)a.M, (int)a.N, (int)a.K, (int)a.P, a.ep);
  return hipGetLastError();
}

// Groups of 32 channels and four waves where a CU gets two of them, else smaller groups and more waves.
template <int MT, int XDT>
hipError_t run_m(const MxArgs& a, const DeviceCaps& caps, hipStream_t st) {
  if (a.N < 2 * 32 * (int64_t)caps.cus) return a.P <= 4096 ? run<8, 1, 2, MT, XDT, 4>(a, caps, st) : run<8, 1, 3, MT, XDT, 12>(a, caps, st);
  return a.P <= 4096 ? run<4, 2, 3, MT, XDT, 8>(a, caps, st) : run<4, 2, 3, MT, XDT, 16>(a, caps, st);
}
template <int XDT>
hipError_t run_x(const MxArgs& a, const DeviceCaps& caps, hipStream_t st) {
  return a.M <= 4 ? run_m<4, XDT>(a, caps, st) : run_m<kMaxM, XDT>(a, caps, st);
}

// Up to 16 CT tokens whose codes are ready: as above, but a unit in the ring also holds the tokens' rows,
// read again for each group of 16 RT channels (they stay in the L2s).  No split planes, no second launch:
// 32 tokens at (N, K) = (4096, 11008) 9.5 us, on tiles and a sum of splits 11.8; (4096, 4096) 5.4, 8.2; 24
// tokens at (16384, 16384) 35.0, 38.0.
template <int NW, int RT, int CT, int SLOTS>
__global__ __launch_bounds__(NW * 64) void mx_few_kernel(const uint8_t* __restrict__ W, const uint8_t* __restrict__ we,
                                                         const uint8_t* __restrict__ A, const uint8_t* __restrict__ ae, int M,
                                                         int N, int P, const Epi ep) {
  constexpr int T = NW * 64, nD = 2 * (RT + CT) + 2;  // loads of a unit
  constexpr int EXPS = (RT + CT) * 2048, SLOT = EXPS + 512;
  static_assert(RT <= 2 && CT <= 2, "exponents of 32 rows by a load");
  extern __shared__ __attribute__((aligned(16))) char smem[];  // rings [NW][SLOTS][SLOT]
  __shared__ float sums[2][NW][RT * 16][CT * 16 + 1];          // of groups in turn
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int units = (P + 255) >> 8, groups = (N + RT * 16 - 1) / (RT * 16);
  const int row = P >> 1, erow = P >> 5;  // bytes of a row's codes and exponents
  const int r16 = lane & 15, q4 = lane >> 4;
  char* own = smem + wave * (SLOTS * SLOT);
  int off[2];  // where a lane's loads of 8 rows begin
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = 8 * j + (lane >> 3);
    off[j] = r * row + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
  }
  const int eoff = (lane >> 1) * erow + (lane & 1) * 4;
  // A group of channels and the unit (one step also where the wave has none).
  struct Place {
    int group, u;
  };
  auto advance = [&](Place& p) {
    p.u += NW;
    if (p.u < units) return;
    p.u = wave;
    p.group += gridDim.x;
  };
  // channels and tokens past the last one, and all of a place past the end: 0, without a request
  auto load = [&](const Place& p, int slot) {
    char* at = own + slot * SLOT;
    const bool in = p.group < groups && p.u < units;
    const size_t n0 = (size_t)p.group * (RT * 16);
    const int rows = in ? min(RT * 16, N - (int)n0) : 0, tokens = in ? M : 0;
#pragma unroll
    for (int r = 0; r < RT + CT; ++r) {
      const uint8_t* base = r < RT ? W + (n0 + r * 16) * row : A + (size_t)((r - RT) * 16) * row;
      const int left = r < RT ? rows - r * 16 : tokens - (r - RT) * 16;
      const rsrc_t rs = mx_rsrc(base, __builtin_amdgcn_readfirstlane(max(0, min(left, 16)) * (uint32_t)row));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        char* to = at + r * 2048 + j * 1024;
        if (r < RT) __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)to, 16, (int)off[j], (int)(p.u * 128), 0, kNonTemporal);
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)to, 16, (int)off[j], (int)(p.u * 128), 0, 0);
      }
    }
    const rsrc_t re = mx_rsrc(we + n0 * erow, __builtin_amdgcn_readfirstlane(rows * (uint32_t)erow));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(re, (lds_void*)(at + EXPS), 4, (int)eoff, (int)(p.u * 8), 0, 0);
    const rsrc_t ra = mx_rsrc(ae, __builtin_amdgcn_readfirstlane(tokens * (uint32_t)erow));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(at + EXPS + 256), 4, (int)eoff, (int)(p.u * 8), 0, 0);
  };
  Place now = {(int)blockIdx.x, wave}, ahead = now;
#pragma unroll
  for (int k = 0; k < SLOTS - 1; ++k) {
    load(ahead, k);
    advance(ahead);
  }
  f32x4 acc[RT][CT];
  auto begin = [&]() {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  begin();
  int slot = 0, turn = 0;
  while (now.group < groups) {
    load(ahead, slot == 0 ? SLOTS - 1 : slot - 1);
    advance(ahead);
    {
      constexpr int n = (SLOTS - 1) * nD;
      static_assert(n < 64, "the wait's counter");
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt((n & 15) | 0xF70 | ((n >> 4) << 14));
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    }
    if (now.u < units) {
      const char* at = own + slot * SLOT;
      u32x2 ew[RT], ex[CT];
#pragma unroll
      for (int r = 0; r < RT; ++r) ew[r] = *reinterpret_cast<const u32x2*>(at + EXPS + (r * 16 + r16) * 8);
#pragma unroll
      for (int c = 0; c < CT; ++c) ex[c] = *reinterpret_cast<const u32x2*>(at + EXPS + 256 + (c * 16 + r16) * 8);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && now.u * 256 + 128 >= P) break;  // the row ends in the middle of its last unit
        const int chunk = r16 * 128 + (((4 * h + q4) ^ (r16 >> 1)) << 4);
        u32x4 x[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) x[c] = *reinterpret_cast<const u32x4*>(at + (RT + c) * 2048 + chunk);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const u32x4 w = *reinterpret_cast<const u32x4*>(at + r * 2048 + chunk);
#pragma unroll
          for (int c = 0; c < CT; ++c)
            acc[r][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(w), mx_operand(x[c]), acc[r][c], kFp4, kFp4, 0,
                                                                         (int)(ew[r][h] >> (8 * q4)), 0, (int)(ex[c][h] >> (8 * q4)));
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    slot = slot == SLOTS - 1 ? 0 : slot + 1;
    if (now.u + NW >= units) {
      // the group's sums, by waves in turn, with one barrier a group (as above)
      float(*sum)[RT * 16][CT * 16 + 1] = sums[turn & 1];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[wave][r * 16 + q4 * 4 + i][c * 16 + r16] = acc[r][c][i];
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      for (int i = ((wave + turn) & (NW - 1)) * 64 + lane; i < M * (RT * 16); i += T) {
        const int m = i / (RT * 16), c = i % (RT * 16), n = now.group * (RT * 16) + c;
        if (n >= N) continue;
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NW; ++v) s += sum[v][c][m];
        epi_put(ep, epi_col(ep, n), m, s);
      }
      ++turn;
      begin();
    }
    advance(now);
  }
  __builtin_amdgcn_s_waitcnt(0x0070);  // no direct LDS load may land after the workgroup's LDS is handed on
}

template <int NW, int RT, int CT, int SLOTS>
hipError_t run_few(const MxArgs& a, const DeviceCaps& caps, hipStream_t st) {
  static_assert((NW & (NW - 1)) == 0, "waves in turn");
  constexpr int lds = NW * SLOTS * ((RT + CT) * 2048 + 512), fixed = 2 * NW * RT * 16 * (CT * 16 + 1) * 4;
  static_assert(lds + fixed <= 160 * 1024, "a CU's LDS");
  auto k = mx_few_kernel<NW, RT, CT, SLOTS>;
  if (lds + fixed > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int64_t groups = (a.N + RT * 16 - 1) / (RT * 16), per_cu = 160 * 1024 / (lds + fixed);
  k<<<(unsigned)std::min<int64_t>(groups, per_cu * caps.cus), NW * 64, lds, st>>>(a.W, a.w_scales, a.A, a.a_scales, (int)a.M, (int)a.N,
                                                                                (int)a.P, a.ep);
  return hipGetLastError();
}

}  // namespace

bool mx_decode_supported(int64_t M, int64_t K) { return M <= kMaxM && M * mx_pitch(K) <= max_columns(M); }
bool mx_decode_ready_supported(int64_t M, int64_t K) { return M <= kReadyM && mx_decode_supported(M, K); }

// One or two ready tokens are faster where they lie in LDS: (4096, 11008) 6.1 us for one, 6.8 here; from
// three on here: four 7.5, 6.8.
// The waves of a workgroup go through a whole row, so where groups of 16 channels leave half of the CUs idle
// a long one is faster on tiles that split it: (512, 65536) 16 tokens 24.5 us here, 20.9 so, 32 tokens 35.6,
// 23.0; (2048, 32768) 14.8, 16.5 and 20.4, 18.4; (2048, 16384) 8.7, 11.4 and 11.7, 12.5; (128, 4096) 3.9, 6.7
// and 5.0, 7.2.  With more groups it is the other way about, or within a tenth: (3000, 65536) 29.0, 33.2 and 40.4,
// 37.7; (8192, 65536) 61, 70 and 64, 72.
bool mx_few_supported(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps) {
  if (M > kFewM || mx_decode_ready_supported(M, K)) return false;
  return (N + 15) / 16 * 2 > caps.cus || mx_pitch(K) <= (M <= 16 ? 36864 : 18432);
}

// Groups of 32 channels where they make nearly whole rounds of the CUs, else of 16, two workgroups a CU
// (twice the tokens' reads): 16 tokens at (8192, 8192) 10.6 us, 11.6 of 16; at (11008, 4096), 1.3 rounds, 9.0,
// 8.3.  Tiles for as many: 13.1 and 9.1.
hipError_t launch_mx_few(const MxArgs& a, const DeviceCaps& caps, hipStream_t st) {
  const int64_t groups = (a.N + 31) / 32, rounds = (groups + caps.cus - 1) / caps.cus;
  if (groups * 5 >= rounds * caps.cus * 4) return a.M <= 16 ? run_few<4, 2, 1, 3>(a, caps, st) : run_few<4, 2, 2, 3>(a, caps, st);
  return a.M <= 16 ? run_few<4, 1, 1, 3>(a, caps, st) : run_few<4, 1, 2, 2>(a, caps, st);
}

hipError_t launch_mx_decode(const MxArgs& a, const DeviceCaps& caps, hipStream_t st) {
  if (a.X == nullptr) return run_m<kReadyM, -1>(a, caps, st);
  switch (a.x_dt) {
    case W4_DT_F32: return run_x<W4_DT_F32>(a, caps, st);
    case W4_DT_F16: return run_x<W4_DT_F16>(a, caps, st);
    default: return run_x<W4_DT_BF16>(a, caps, st);
  }
}

}  // namespace w4
