// Product of microscaled 4-bit rows for one to sixteen tokens (decode), for gfx950.  The weight is read
// once, and its bytes set the time; float tokens are quantized by the same launch.
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
constexpr int kMaxM = 16;             // tokens
// Columns of all tokens.  Every workgroup quantizes them, and past these the tiles behind a launch that
// quantizes once are as fast: (N, K) = (12288, 4096), 8 tokens 10.1 us here, 11.9 on the tiles, 12
// tokens 13.1 and 12.1; (4096, 11008), 4 tokens 8.4, 13.0, 8 tokens 14.8, 13.7; (16384, 16384), 2 tokens
// 32.4, 36.3, 4 tokens 39.6, 36.4.
constexpr int64_t kMaxColumns = 45056;

// The tokens in LDS: exponents [M][P / 32], then codes [M][P / 2 + 16] (the pad keeps the tokens' rows in
// distinct banks).
constexpr int codes_at(int64_t M, int64_t P) { return (int)((M * (P >> 5) + 15) & ~(int64_t)15); }
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
  const int at_codes = codes_at(M, P);

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
        if ((c & 3) == 0) tokens[m * erow + (c >> 2)] = (char)e;
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
        *reinterpret_cast<uint32_t*>(tokens + m * erow + c * 4) = *reinterpret_cast<const uint32_t*>(ae + (size_t)m * erow + c * 4);
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
  const char* xe = tokens + m0 * erow;
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

}  // namespace

bool mx_decode_supported(int64_t M, int64_t K) { return M <= kMaxM && M * mx_pitch(K) <= kMaxColumns; }

hipError_t launch_mx_decode(const MxArgs& a, const DeviceCaps& caps, hipStream_t st) {
  if (a.X == nullptr) return run_x<-1>(a, caps, st);
  switch (a.x_dt) {
    case W4_DT_F32: return run_x<W4_DT_F32>(a, caps, st);
    case W4_DT_F16: return run_x<W4_DT_F16>(a, caps, st);
    default: return run_x<W4_DT_BF16>(a, caps, st);
  }
}

}  // namespace w4
