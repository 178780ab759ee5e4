// A mixture-of-experts layer on microscaled 4-bit weights for a few tokens (mx4_moe), for gfx950.
// For token t with logits z over E experts, j over the `top` largest (by value, then lower index):
//   g_j = exp(z_j - max z) / total,  total over the chosen (renormalized) or over all experts
//   a_j = silu(W1g[j] x) * (W1u[j] x),  y = sum_j g_j W2[j] a_j
// in two launches: the choice of experts and g_j a_j, then the sum over experts (and, where the
// rows of y alone would leave compute units idle, a third that adds its parts).
//
// What bounds it: the weights of the experts that some token reaches, each read once.  A wave has its own
// ring of units in LDS, filled by direct loads (in registers their lanes, each at a row of its own,
// cost the vector caches a tag for every 16 bytes); they are widened to bf16 (exactly: two significant
// bits) and multiplied on the matrix cores with up to sixteen tokens as the columns.  The activations
// enter as bf16 parts whose sum they are (one of bf16, two of fp16, three of fp32), and so does g_j a_j
// (three of an fp32): the matrix cores have time for it, and nothing is rounded between the products.  (Two
// parts, 16 bits, lose differences of nearly equal activations; in a captured graph 173 us instead of 196 for
// 32 tokens, 2 of 8 experts of 4096 x 11008, sixteen columns a product; of four, 77.0 and 78.6 for 4 tokens.)
// Launches, bf16: 4 tokens, 2 of 8 experts of 4096 x 11008, 43-50 us (262 MB, 5.3-6.2 TB/s), 31-35 (131 MB),
// 4.8 for the parts; 32 tokens, 8 of 128 experts of 2048 x 768, 46 (187 MB), 25 and 4.6.  Reads of the
// same pattern alone reach 5.7-6.4 TB/s; the rest is the choice ahead of the first weight (some 5 us for
// 32 tokens) and the ends of the launches.  One token, 8 of 128 experts: 10.7 and 7.5, all latency.
#include <algorithm>

#include "api_common.h"
#include "launch.h"
#include "mx.h"

namespace w4 {

namespace {

constexpr int kNonTemporal = 2;  // cache-policy operand of a load
constexpr int kTokens = kMoeTokens, kMaxTop = kMoeTop, kMaxExperts = kMoeExperts;
constexpr int kNone = 0x7FFF0000;  // a buffer offset that is out of range: 0 without a request
constexpr int NW = 4;              // waves of a workgroup; a CU holds two workgroups

// The experts that the tokens reach, in the order of their numbers, as the second launch takes them
// from the workspace: expert, its tokens' number and first row of g_j a_j, and the rows' tokens.
struct Reached {
  uint64_t bad;  // tokens whose logits hold a NaN or +infinity
  int count;
  uint16_t expert[kMaxExperts], first[kMaxExperts];
  uint8_t cols[kMaxExperts], token[kTokens * kMaxTop];
};

// What a workgroup of the first launch holds of the choice, and what it needs while it makes it.
struct Routing : Reached {
  float gate[kTokens * kMaxTop];  // g_j of each row
};
struct Choice {
  uint64_t tokens[kMaxExperts];  // of each expert
  float weight[kTokens][kMaxTop];
  short chosen[kTokens][kMaxTop];
  short slot[kMaxExperts];  // of each expert that is reached
};

// Maximum, minimum and sum over a row of sixteen lanes, in every lane of it.
template <typename F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, int none, F f) {  // f(v, none) = v
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(none, (int)v, 0x140, 0xF, 0xF, false));  // row mirror
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(none, (int)v, 0x141, 0xF, 0xF, false));  // half-row mirror
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(none, (int)v, 0x4E, 0xF, 0xF, false));   // lane ^ 2
  return f(v, (uint32_t)__builtin_amdgcn_update_dpp(none, (int)v, 0xB1, 0xF, 0xF, false));  // lane ^ 1
}
__device__ __forceinline__ uint32_t row_umax(uint32_t v) {
  return row_reduce(v, 0, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint32_t row_umin(uint32_t v) {
  return row_reduce(v, -1, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
__device__ __forceinline__ float row_sum(float v) {
  return __uint_as_float(row_reduce(__float_as_uint(v), 0, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

__device__ __forceinline__ float logit(const void* z, int dt, int64_t i) {
  if (dt == W4_DT_F32) return static_cast<const float*>(z)[i];
  const uint32_t b = static_cast<const uint16_t*>(z)[i];
  return dt == W4_DT_F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
}

// Values as unsigned integers of the same order.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The largest of C keys.
template <int C>
__device__ __forceinline__ uint32_t largest(const uint32_t (&key)[C]) {
  uint32_t m = key[0];
#pragma unroll
  for (int c = 1; c < C; ++c) m = umax(m, key[c]);
  return m;
}

// The choice for four tokens at a time, a row of sixteen lanes each (from token t0; none past T): lane l
// of a row holds experts l C .. l C + C - 1, and the largest is taken out `top` times, the one of the
// lowest number among equals; lane j keeps choice j.
// A round is short where a key says which expert it is: its last nine bits give way to the number, the
// lower the larger.  16-bit logits lose nothing by it.  Of fp32 logits it may not tell the last choice
// from the next one, and where these agree in the bits left the choice is made again with whole keys.
// (Whole keys throughout: 19.6 us instead of 18.9 for a call of one token and 8 of 128 experts.)
template <int C>
__device__ __forceinline__ void choose(Routing& s, Choice& c0, const void* __restrict__ logits, int ldt, int64_t ldl, int t0,
                                       int T, int E, int top, bool renorm) {
  constexpr uint32_t kNumber = kMaxExperts - 1;
  static_assert((kMaxExperts & kNumber) == 0, "bits of a number");
  const int l16 = threadIdx.x & 15, t = t0 + ((threadIdx.x & 63) >> 4), first = l16 * C;
  const uint32_t masked = order_key(-__builtin_inff());  // (its last nine bits are ones)
  uint32_t key[C];
  float v[C];
#pragma unroll
  for (int c = 0; c < C; ++c) v[c] = t < T && first + c < E ? logit(logits, ldt, t * ldl + first + c) : -__builtin_inff();
  uint32_t odd = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    odd |= !(v[c] < __builtin_inff()) ? 1u : 0u;
    key[c] = order_key(v[c] + 0.0f);  // -0 and +0 are equal
  }
  odd = row_umax(odd);
  const uint32_t most = row_umax(largest<C>(key));
  const float mx = most <= masked ? 0.0f : __uint_as_float(most & 0x80000000u ? most & 0x7FFFFFFFu : ~most);
#pragma unroll
  for (int c = 0; c < C; ++c) key[c] = (key[c] & ~kNumber) | (kNumber - (uint32_t)(first + c));
  int chosen = -1;
  uint32_t best = 0;
  for (int j = 0; j < top; ++j) {
    best = row_umax(largest<C>(key));
#pragma unroll
    for (int c = 0; c < C; ++c) key[c] = key[c] == best ? 0u : key[c];
    if (l16 == j && best > masked) chosen = (int)(kNumber - (best & kNumber));
  }
  bool unclear = false;
  if (ldt == W4_DT_F32) {
    const uint32_t next = row_umax(largest<C>(key));
    unclear = next > masked && (next & ~kNumber) == (best & ~kNumber);
  }
  if (__ballot(unclear) != 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) key[c] = order_key(v[c] + 0.0f);
    for (int j = 0; j < top; ++j) {
      best = row_umax(largest<C>(key));
      uint32_t at = 0xFFFFu;
#pragma unroll
      for (int c = C - 1; c >= 0; --c) at = key[c] == best ? (uint32_t)(first + c) : at;
      at = row_umin(at);
#pragma unroll
      for (int c = 0; c < C; ++c) key[c] = at == (uint32_t)(first + c) ? 0u : key[c];
      if (l16 == j) chosen = best > masked ? (int)at : -1;
    }
  }
  if (t >= T) chosen = -1;
  const float z = chosen >= 0 ? logit(logits, ldt, t * ldl + chosen) : -__builtin_inff();
  const float weight = expf(z - mx);  // 0 where there is none
  float sum = weight;
  if (!renorm) {
    sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) sum += expf(v[c] - mx);
  }
  const float total = row_sum(sum);
  if (t >= T) return;
  if (odd != 0) {
    if (l16 == 0) atomicOr(reinterpret_cast<unsigned long long*>(&s.bad), 1ull << t);
    chosen = -1;
  }
  if (l16 < top) {
    c0.chosen[t][l16] = (short)chosen;
    c0.weight[t][l16] = weight / total;
    if (chosen >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&c0.tokens[chosen]), 1ull << t);
  }
}

// This wave's LDS reads and writes done, then a barrier with no fence (a fence would wait for the
// weights in flight).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Every workgroup makes the choice for all tokens.
__device__ __forceinline__ void route(Routing& s, Choice& c, const void* __restrict__ logits, int ldt, int64_t ldl, int T, int E,
                                      int top, bool renorm) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int e = tid; e < E; e += NW * 64) c.tokens[e] = 0;
  if (tid == 0) s.bad = 0;
  lds_barrier();
  for (int t = wave * 4; t < T; t += NW * 4) {
    if (E <= 64) choose<4>(s, c, logits, ldt, ldl, t, T, E, top, renorm);
    else if (E <= 128) choose<8>(s, c, logits, ldt, ldl, t, T, E, top, renorm);
    else choose<kMaxExperts / 16>(s, c, logits, ldt, ldl, t, T, E, top, renorm);
  }
  lds_barrier();
  if (wave == 0) {
    int count = 0, rows = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane, n = e < E ? __popcll(c.tokens[e]) : 0;
      const uint64_t live = __ballot(n != 0);
      int upto = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(upto, d, 64);
        if (lane >= d) upto += up;
      }
      if (n != 0) {
        const int at = count + __popcll(live & ((1ull << lane) - 1));
        s.expert[at] = e;
        s.cols[at] = n;
        s.first[at] = rows + upto - n;
        c.slot[e] = (short)at;
      }
      count += __popcll(live);
      rows += __shfl(upto, 63, 64);
    }
    if (lane == 0) s.count = count;
  }
  lds_barrier();
  for (int i = tid; i < T * top; i += NW * 64) {
    const int t = i / top, j = i - t * top, e = c.chosen[t][j];
    if (e < 0) continue;
    const int row = s.first[c.slot[e]] + __popcll(c.tokens[e] & ((1ull << t) - 1));
    s.token[row] = (uint8_t)t;
    s.gate[row] = c.weight[t][j];
  }
  lds_barrier();
}

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A unit: 256 columns of RT tiles of 16 weight rows, 128 bytes and 8 exponents a row.  In LDS, a row's
// 16-byte chunks (a block of 32 columns each) are at chunk ^ (row / 2 % 8), on the source address of
// the direct loads, so that reads of 16 rows hit distinct banks; behind them the exponents, 8 bytes
// a row in groups of 64 words.
constexpr int RT = 2, kSlots = 3;

constexpr int kSlot = RT * 2048 + 256;
constexpr int column_bytes(int parts, int cols) { return cols == 4 ? parts * 2048 : 0; }  // in LDS, of a wave

// Where a lane's direct loads begin: in 16 rows of codes by two loads of 8 rows, and in the exponents of
// twice 16 rows, the second sixteen `apart` rows behind the first.
struct Lanes {
  int codes[2], exponents;
  __device__ __forceinline__ Lanes(int P, int lane, int apart) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 8 * j + (lane >> 3);
      codes[j] = r * (P >> 1) + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
    }
    exponents = ((lane >> 5) * apart + ((lane & 31) >> 1)) * (P >> 5) + (lane & 1) * 4;
  }
};

// Direct loads of 16 rows (those from `rows` on: 0, without a request), unit u, to LDS.
__device__ __forceinline__ void dma_codes(char* at, const uint8_t* W, uint32_t rows, int P, int u, const Lanes& l) {
  const rsrc_t rw = mx_rsrc(W, __builtin_amdgcn_readfirstlane(rows * (uint32_t)(P >> 1)));  // else a loop over lanes
#pragma unroll
  for (int j = 0; j < 2; ++j)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(at + j * 1024), 16, (int)l.codes[j], (int)(u * 128), 0,
                                             kNonTemporal);
}
// The exponents of both sixteens, of `rows` rows in all from the first.
__device__ __forceinline__ void dma_exponents(char* at, const uint8_t* we, uint32_t rows, int P, int u, const Lanes& l) {
  const rsrc_t re = mx_rsrc(we, __builtin_amdgcn_readfirstlane(rows * (uint32_t)(P >> 5)));
  __builtin_amdgcn_raw_ptr_buffer_load_lds(re, (lds_void*)at, 4, (int)l.exponents, (int)(u * 8), 0, 0);
}

// A unit's columns for up to COLS tokens, NP bf16 parts `step` bytes after one another, on their way in
// registers; lane l multiplies blocks l / 16 and 4 + l / 16 of eight for column l % 16.
// COLS = 16: as they are multiplied.  COLS = 4 (eight loads would fetch mostly nothing, and the caches'
// return path is what the weights need as well: 108 us with them, 96 without, 4 tokens on 2 of 8 experts
// of 4096 x 11008): rows of four tokens by two loads a part, through LDS (put, [NP][4][512 bytes], the
// 16-byte chunks of part k of token t at chunk ^ (t + 4 k), so that most reads hit distinct banks), and the parts
// are columns of their own, 4 k + t of sixteen: one product takes all of them, and join adds their sums.
template <int NP, int COLS>
struct Columns {
  u32x4 x[NP][COLS == 4 ? 2 : 8];

  // row(c): byte offset of token c's columns, kNone for no token; `width` columns lie in a row
  template <typename F>
  __device__ __forceinline__ void fetch(rsrc_t rx, F row, int u, int width, int step, int lane) {
    if constexpr (COLS == 4) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = 2 * j + (lane >> 5), chunk = (lane & 31) ^ t, col = u * 256 + chunk * 8, r = row(t);
        const int at = r != kNone && col < width ? r + col * 2 : kNone;
#pragma unroll
        for (int k = 0; k < NP; ++k) x[k][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, at, k * step, 0));
      }
    } else {
      const int col = u * 256 + (lane >> 4) * 32, r = row(lane & 15);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = r != kNone && col + h * 128 < width ? r + (col + h * 128) * 2 : kNone;
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[k][h * 4 + i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, at + i * 16, k * step, 0));
      }
    }
  }
  __device__ __forceinline__ void put(char* xs, int lane) const {
    if constexpr (COLS == 4) {
#pragma unroll
      for (int k = 0; k < NP; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) *reinterpret_cast<u32x4*>(xs + k * 2048 + j * 1024 + (lane ^ 4 * k) * 16) = x[k][j];
    }
  }
  // the operands of a product: parts [kOperands] of a column, or the part that a column is
  static constexpr int kOperands = COLS == 4 ? 1 : NP;
  __device__ __forceinline__ u32x4 operand(const char* xs, int k, int h, int i, int lane) const {
    if constexpr (COLS == 4) {
      const int t = lane & 3, p = min((lane & 15) >> 2, NP - 1);  // columns past the parts: not used
      return *reinterpret_cast<const u32x4*>(xs + p * 2048 + t * 512 + ((((4 * h + (lane >> 4)) * 4 + i) ^ (t + 4 * p)) << 4));
    } else {
      return x[k][h * 4 + i];
    }
  }
  // a column's sum in the lane of that column
  __device__ __forceinline__ static f32x4 join(const f32x4& v) {
    f32x4 s = v;
    if constexpr (COLS == 4 && NP > 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v[i]), 0x104, 0xF, 0xF, false));  // lane + 4
        if constexpr (NP > 2)
          s[i] += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v[i]), 0x108, 0xF, 0xF, false));  // lane + 8
      }
    }
    return s;
  }
};

// acc[r] += tile r of the unit at `base` times the columns.  whole: the unit's second half lies in the
// row, too.
// The conversion takes its power from the exponent bits of an fp32 alone (checked over all exponents,
// 0 and NaN's among them, with any sign and mantissa): byte q4 of a word is rotated there.
template <int NP, int COLS>
__device__ __forceinline__ void multiply(const char* base, const Columns<NP, COLS>& c, const char* xs, bool whole, int lane,
                                         f32x4 (&acc)[RT]) {
  const int r16 = lane & 15, q4 = lane >> 4;
  u32x4 w[2][RT];
  u32x2 e[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h][r] = *reinterpret_cast<const u32x4*>(base + r * 2048 + r16 * 128 + (((4 * h + q4) ^ (r16 >> 1)) << 4));
    e[r] = *reinterpret_cast<const u32x2*>(base + RT * 2048 + r * 128 + r16 * 8);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h == 1 && !whole) break;
    float p[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) p[r] = __uint_as_float(__builtin_amdgcn_alignbit(e[r][h], e[r][h], 8 * q4 + 9));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 a[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) a[r] = mx_bf16x8(w[h][r][i], p[r]);
#pragma unroll
      for (int k = 0; k < Columns<NP, COLS>::kOperands; ++k) {
        const u32x4 x = c.operand(xs, k, h, i, lane);
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = mfma16(a[r], x, acc[r]);
      }
    }
  }
}

// All loads but the last n done.
template <int n>
__device__ __forceinline__ void wait_loads() {
  static_assert(n < 64, "the wait's counter");
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((n & 15) | 0xF70 | ((n >> 4) << 14));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// First launch: the choice, then items of 16 gate rows and the same up rows of one expert, for COLS of its
// tokens at a time, whose contraction the workgroup's waves share.  While a wave multiplies a
// unit, the columns of the next and the weights of the next two, of this item or those that follow,
// are on their way, also while an item's sums are put together.
// x [T][NP][ldx] bf16 parts, Hx (a multiple of 32) columns of each to read; a [rows][HP][Fp] bf16
// parts of g_j a_j, a row for each expert and token of it.
template <int DT, int COLS>
__global__ __launch_bounds__(NW * 64) void moe_up_kernel(const uint16_t* __restrict__ x, int ldx, int Hx,
                                                         const void* __restrict__ logits, int ldt, int64_t ldl,
                                                         const uint8_t* __restrict__ W, const uint8_t* __restrict__ we, int T,
                                                         int E, int top, int renorm, int P, int F, int Fp,
                                                         uint16_t* __restrict__ a, Reached* __restrict__ reached) {
  constexpr int NP = mx_parts(DT), HP = kMoeParts;
  constexpr int nD = 5, nX = COLS == 4 ? NP * 2 : NP * 8;  // loads of a unit's weights and columns
  extern __shared__ __attribute__((aligned(16))) char ring[];  // [NW][kSlots][kSlot], then columns [NW][column_bytes]
  __shared__ Routing s;
  __shared__ __attribute__((aligned(16))) float sums[2][NW][RT * 16][COLS + 1];  // of items in turn
  static_assert(sizeof(Choice) <= NW * kSlots * kSlot, "the choice is made where the ring will be");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  route(s, *reinterpret_cast<Choice*>(ring), logits, ldt, ldl, T, E, top, renorm != 0);
  const int count = __builtin_amdgcn_readfirstlane(s.count);
  if (blockIdx.x == 0) {  // for the second launch
    for (int i = tid; i < count; i += NW * 64) {
      reached->expert[i] = s.expert[i];
      reached->cols[i] = s.cols[i];
      reached->first[i] = s.first[i];
    }
    for (int i = tid; i < T * top; i += NW * 64) reached->token[i] = s.token[i];
    if (tid == 0) {
      reached->count = count;
      reached->bad = s.bad;
    }
  }
  const int tiles = Fp / 16;
  if ((int)blockIdx.x >= count * tiles) return;
  const int units = (P + 255) >> 8;  // wave w takes units w, w + NW, ..
  const rsrc_t rx = mx_rsrc(x, (uint32_t)T * (uint32_t)(NP * ldx) * 2u);
  char* own = ring + wave * (kSlots * kSlot);
  char* xs = ring + NW * kSlots * kSlot + wave * column_bytes(NP, COLS);

  // An item (a tile of the expert in a slot), the tokens of its expert from b0, the unit (one step also
  // where the wave has none), and the item's gate rows (`rows` that are to be read).
  struct Place {
    int slot, tile, b0, u, cols, first;
    uint32_t rows;
    const uint8_t *w, *e;
  };
  const size_t codes_up = (size_t)F * (P >> 1);
  auto enter = [&](Place& p) {
    const int e = __builtin_amdgcn_readfirstlane(s.expert[p.slot]), f0 = p.tile * 16;
    p.cols = __builtin_amdgcn_readfirstlane(s.cols[p.slot]);
    p.first = __builtin_amdgcn_readfirstlane(s.first[p.slot]);
    p.rows = wave < units ? (uint32_t)max(0, min(16, F - f0)) : 0u;
    const size_t g = (size_t)e * 2 * F + f0;
    p.w = W + g * (P >> 1);
    p.e = we + g * (P >> 5);
  };
  const int more_slots = gridDim.x / (unsigned)tiles, more_tiles = gridDim.x - more_slots * tiles;
  auto advance = [&](Place& p) {
    if (p.u + NW < units) {
      p.u += NW;
      return;
    }
    p.u = wave;
    p.b0 += COLS;
    if (p.b0 < p.cols) return;
    p.b0 = 0;
    p.slot += more_slots;
    p.tile += more_tiles;
    if (p.tile >= tiles) {
      p.tile -= tiles;
      ++p.slot;
    }
    if (p.slot < count) enter(p);
    else p.rows = 0u, p.cols = 0;
  };
  const Lanes lanes(P, lane, F);
  auto load = [&](const Place& p, int slot) {
    char* at = own + slot * kSlot;
    dma_codes(at, p.w, p.rows, P, p.u, lanes);
    dma_codes(at + 2048, p.w + codes_up, p.rows, P, p.u, lanes);
    // (gate rows past the last get up rows' exponents: with codes 0, and their sums are not used)
    dma_exponents(at + RT * 2048, p.e, p.rows > 0 ? F + p.rows : 0u, P, p.u, lanes);
  };
  auto columns = [&](Columns<NP, COLS>& c, const Place& p) {
    c.fetch(rx, [&](int t) {
      return p.u < units && p.b0 + t < p.cols ? (int)s.token[p.first + p.b0 + t] * (NP * ldx * 2) : kNone;
    }, p.u, Hx, ldx * 2, lane);
  };
  f32x4 acc[RT];
  auto begin = [&]() {
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  // Sums of the waves, activation, weight, and the parts (as of mx_parts_kernel: the rest cut to eight
  // bits), by waves in turn.  One barrier an item: the next item's sums have a
  // place of their own, and when they are written every wave has passed this one's.
  int turn = 0;
  auto finish = [&](const Place& p) {
    float(*sum)[RT * 16][COLS + 1] = sums[turn & 1];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = Columns<NP, COLS>::join(acc[r]);
    if ((lane & 15) < COLS) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[wave][r * 16 + (lane >> 4) * 4 + i][lane & 15] = acc[r][i];
    }
    lds_barrier();
    const int f = lane & 15, c = ((wave + turn) & (NW - 1)) * 4 + (lane >> 4), col = p.b0 + c;
    ++turn;
    static_assert(NW == 4, "sixteen tokens, four a wave");
    if (c < COLS && col < p.cols) {
      float g = 0.0f, up = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        g += sum[v][f][c];
        up += sum[v][16 + f][c];
      }
      float v = p.tile * 16 + f < F ? g / (1.0f + expf(-g)) * up * s.gate[p.first + col] : 0.0f;
      uint16_t* o = a + (size_t)(p.first + col) * (HP * Fp) + p.tile * 16 + f;
      const bool odd = (__float_as_uint(v) & 0x7FFFFFFFu) >= 0x7F800000u;
#pragma unroll
      for (int k = 0; k < HP; ++k) {
        uint32_t bits = __float_as_uint(v) >> 16;
        if (odd) bits = k > 0 ? 0u : (__float_as_uint(v) & 0x7FFFFFu) != 0 ? 0x7FC0u : bits;
        o[(size_t)k * Fp] = (uint16_t)bits;
        v -= __uint_as_float(bits << 16);
        if (odd) v = 0.0f;
      }
    }
  };
  Place now, next, after;  // of the products, the columns, the weights
  now.slot = blockIdx.x / (unsigned)tiles;
  now.tile = blockIdx.x - now.slot * tiles;
  now.b0 = 0;
  now.u = wave;
  enter(now);
  load(now, 0);
  next = now;
  advance(next);
  Columns<NP, COLS> c0, c1;
  columns(c0, now);
  load(next, 1);
  after = next;
  advance(after);
  begin();
  c0.put(xs, lane);
  int slot = 0;
  auto step = [&](const Columns<NP, COLS>& c, Columns<NP, COLS>& coming) {
    const int spare = slot == 0 ? kSlots - 1 : slot - 1;
    columns(coming, next);
    load(after, spare);
    wait_loads<2 * nD + nX>();
    if (now.u < units) multiply<NP, COLS>(own + slot * kSlot, c, xs, now.u * 256 + 128 < P, lane, acc);
    __builtin_amdgcn_sched_barrier(0);
    slot = slot == kSlots - 1 ? 0 : slot + 1;
    if (now.u + NW >= units) {
      finish(now);
      begin();
    }
    coming.put(xs, lane);
    now = next;
    next = after;
    advance(after);
    return now.slot < count;
  };
  while (step(c0, c1) && step(c1, c0)) {
  }
  wait_loads<0>();  // no direct LDS load may land after the workgroup's LDS is handed on
}

template <int DT>
__device__ __forceinline__ void store(void* out, int64_t i, float v) {
  if constexpr (DT == W4_DT_F32) static_cast<float*>(out)[i] = v;
  else if constexpr (DT == W4_DT_BF16) static_cast<uint16_t*>(out)[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
  else static_cast<uint16_t*>(out)[i] = f32_to_f16_bits(v);
}

// Second launch: 32 rows of y for a workgroup, whose waves share the units of all reached experts with
// those of the other S - 1 workgroups of these rows.  The columns are COLS of an expert's tokens; at
// the end of its units a wave adds them to its own sums of all tokens in LDS, [T][32].  (Columns for
// all tokens, 0 for those without the expert, would need no LDS but read and multiply zeros, and a
// NaN among the weights would reach every token.)
constexpr int kRowPitch = RT * 16 + 4;

template <int DT, int COLS, int SLOTS, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void moe_down_kernel(const uint16_t* __restrict__ a, const Reached* __restrict__ reached,
                                                           const uint8_t* __restrict__ W, const uint8_t* __restrict__ we, int T,
                                                           int E, int top, int H, int Fp, int S, void* __restrict__ out,
                                                           int64_t ldo, float* __restrict__ part) {
  constexpr int HP = kMoeParts;
  constexpr int nD = 5, nX = COLS == 4 ? HP * 2 : HP * 8;  // loads of a unit's weights and columns
  // rings [WAVES][SLOTS][kSlot], columns [WAVES][column_bytes], sums [WAVES][T][kRowPitch], and of Reached
  // as much as there may be: all of it would take the place of the second workgroup on a CU
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float* sums = reinterpret_cast<float*>(smem + WAVES * (SLOTS * kSlot + column_bytes(HP, COLS)));
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int most = min(E, T * top);
  struct {
    uint16_t *expert, *first;
    uint8_t *cols, *token;
  } s;
  s.expert = reinterpret_cast<uint16_t*>(sums + WAVES * T * kRowPitch);
  s.first = s.expert + most;
  s.cols = reinterpret_cast<uint8_t*>(s.first + most);
  s.token = s.cols + most;
  for (int i = tid; i < most; i += WAVES * 64) {  // past the count: not used
    s.expert[i] = reached->expert[i];
    s.cols[i] = reached->cols[i];
    s.first[i] = reached->first[i];
  }
  for (int i = tid; i < T * top; i += WAVES * 64) s.token[i] = reached->token[i];
  const int count = __builtin_amdgcn_readfirstlane(reached->count);
  const uint64_t bad = reached->bad;
  for (int i = tid; i < WAVES * T * kRowPitch; i += WAVES * 64) sums[i] = 0.0f;
  lds_barrier();
  const int group = blockIdx.x / (unsigned)S, slice = blockIdx.x - group * S;
  const int h0 = group * 16 * RT;
  const uint32_t rows = (uint32_t)min(16 * RT, H - h0);
  const int of_expert = (Fp + 255) >> 8, units = count * of_expert;
  const int per = (units + S * WAVES - 1) / (S * WAVES);
  const int u0 = min((slice * WAVES + wave) * per, units), u1 = min(u0 + per, units);
  const rsrc_t rx = mx_rsrc(a, (uint32_t)(T * top) * (uint32_t)(HP * Fp) * 2u);
  float* mine = sums + wave * T * kRowPitch;
  char* own = smem + wave * (SLOTS * kSlot);
  char* xs = smem + WAVES * SLOTS * kSlot + wave * column_bytes(HP, COLS);
  if (u0 < u1) {
    // An expert, its units [from, to) of this wave and the next of them, its tokens from b0.
    struct Place {
      int slot, b0, u, from, to, cols, first;
      uint32_t rows;
      const uint8_t *w, *e;
    };
    const int last_slot = (u1 - 1) / of_expert;
    auto enter = [&](Place& p) {
      const int e = __builtin_amdgcn_readfirstlane(s.expert[p.slot]);
      p.cols = __builtin_amdgcn_readfirstlane(s.cols[p.slot]);
      p.first = __builtin_amdgcn_readfirstlane(s.first[p.slot]);
      p.from = max(u0 - p.slot * of_expert, 0);
      p.to = min(of_expert, u1 - p.slot * of_expert);
      p.u = p.from;
      p.b0 = 0;
      p.rows = rows;
      const size_t first = (size_t)e * H + h0;
      p.w = W + first * (Fp >> 1);
      p.e = we + first * (Fp >> 5);
    };
    auto advance = [&](Place& p) {
      if (++p.u < p.to) return;
      p.u = p.from;
      p.b0 += COLS;
      if (p.b0 < p.cols) return;
      if (++p.slot <= last_slot) enter(p);
      else p.rows = 0u, p.cols = 0;
    };
    const Lanes lanes(Fp, lane, 16);
    auto load = [&](const Place& p, int slot) {
      char* at = own + slot * kSlot;
      dma_codes(at, p.w, p.rows, Fp, p.u, lanes);
      dma_codes(at + 2048, p.w + 16 * (Fp >> 1), p.rows > 16 ? p.rows - 16 : 0u, Fp, p.u, lanes);
      dma_exponents(at + RT * 2048, p.e, p.rows, Fp, p.u, lanes);
    };
    auto columns = [&](Columns<HP, COLS>& c, const Place& p) {
      c.fetch(rx, [&](int t) { return p.b0 + t < p.cols ? (p.first + p.b0 + t) * (HP * Fp * 2) : kNone; }, p.u, Fp, Fp * 2, lane);
    };
    f32x4 acc[RT];
    auto begin = [&]() {
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    Place now, next, after;  // of the products, the columns, the weights
    now.slot = u0 / of_expert;
    enter(now);
    load(now, 0);
    next = now;
    advance(next);
    Columns<HP, COLS> c0, c1;
    columns(c0, now);
    after = next;
    if constexpr (SLOTS == 3) {
      load(next, 1);
      advance(after);
    }
    begin();
    c0.put(xs, lane);
    int slot = 0;
    auto step = [&](const Columns<HP, COLS>& c, Columns<HP, COLS>& coming) {
      const int spare = slot == 0 ? SLOTS - 1 : slot - 1;
      columns(coming, next);
      load(SLOTS == 3 ? after : next, spare);
      wait_loads<(SLOTS - 1) * nD + nX>();
      multiply<HP, COLS>(own + slot * kSlot, c, xs, now.u * 256 + 128 < Fp, lane, acc);
      __builtin_amdgcn_sched_barrier(0);
      slot = slot == SLOTS - 1 ? 0 : slot + 1;
      if (now.u + 1 >= now.to) {
        const int col = now.b0 + (lane & 15);
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = Columns<HP, COLS>::join(acc[r]);
        if ((lane & 15) < COLS && col < now.cols) {
          float* to = mine + s.token[now.first + col] * kRowPitch + (lane >> 4) * 4;
#pragma unroll
          for (int r = 0; r < RT; ++r) *reinterpret_cast<f32x4*>(to + r * 16) += acc[r];
        }
        begin();
      }
      coming.put(xs, lane);
      now = next;
      if constexpr (SLOTS == 3) {
        next = after;
        advance(after);
      } else {
        advance(next);
      }
      return now.slot <= last_slot;
    };
    while (step(c0, c1) && step(c1, c0)) {
    }
    wait_loads<0>();  // no direct LDS load may land after the workgroup's LDS is handed on
  }
  lds_barrier();
  for (int i = tid; i < T * RT * 16; i += WAVES * 64) {
    const int t = i / (RT * 16), h = i - t * (RT * 16);
    if (h >= (int)rows) continue;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < WAVES; ++k) v += sums[(k * T + t) * kRowPitch + h];
    if (part != nullptr) part[((size_t)slice * T + t) * H + h0 + h] = v;
    else store<DT>(out, t * ldo + h0 + h, (bad >> t & 1) != 0 ? __builtin_nanf("") : v);
  }
}

// Third launch, where the rows of y are shared: the parts in their order.
template <int DT>
__global__ __launch_bounds__(256) void moe_join_kernel(const float* __restrict__ part, const Reached* __restrict__ reached, int T,
                                                       int H, int S, void* __restrict__ out, int64_t ldo) {
  const int h = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (h >= H) return;
  float v = 0.0f;
  for (int k = 0; k < S; ++k) v += part[((size_t)k * T + t) * H + h];
  store<DT>(out, t * ldo + h, (reached->bad >> t & 1) != 0 ? __builtin_nanf("") : v);
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Tokens of an expert that its weights are widened for at a time: four where experts have few, else sixteen.
// The choice itself is not known here.  An expert with more than four tokens reads its weights again for
// the next four, but T top <= 3 E bounds that by 3 E / 4 such reads in all, so a batch whose tokens all agree
// costs less than one that reaches every expert: 32 tokens, 8 of 128 experts of 2048 x 768, 55 us and 77; 64,
// 6 of 128, 89 and 106.
bool few_each(const MoeArgs& a) { return a.T <= 4 || a.T * a.top <= 3 * a.E; }

int down_lds(const MoeArgs& a, int cols, int slots, int waves) {
  return waves * (slots * kSlot + column_bytes(kMoeParts, cols) + (int)a.T * kRowPitch * 4) +
         (int)(5 * std::min<int64_t>(a.E, a.T * a.top) + a.T * a.top);
}

// Units of the second launch for the same rows, if all experts that may be reached are.
int64_t down_units(const MoeArgs& a) { return std::min<int64_t>(a.E, a.T * a.top) * ((mx_pitch(a.F) + 255) / 256); }

// Whether one workgroup of eight waves does all of the units of its rows, so that no launch has to join
// parts: where a wave gets few of them.  One token in a captured graph, with the join and without: 22 units
// 22.1 us and 19.3, 36 units 22.9 and 22.0, 48 units 24.5 and 25.0, 64 units 24.7 and 28.4; 4 tokens, 96 units
// 30.2 and 33.5.
bool down_alone(const MoeArgs& a, const DeviceCaps& caps) {
  return few_each(a) && (a.H + RT * 16 - 1) / (RT * 16) <= caps.cus && down_units(a) <= 8 * 6 &&
         down_lds(a, 4, 2, 8) <= 160 * 1024;
}

// Workgroups of the second launch for the same rows: as many as a round of them, two a CU, holds.
int down_slices(const MoeArgs& a, const DeviceCaps& caps) {
  if (down_alone(a, caps)) return 1;
  const int64_t groups = (a.H + RT * 16 - 1) / (RT * 16);
  const int64_t units = down_units(a);
  const int64_t s = std::min<int64_t>(2 * caps.cus / groups, (units + NW - 1) / NW);
  return (int)std::max<int64_t>(1, std::min<int64_t>(s, 16));
}

// The workspace: what the experts reached are, g_j a_j, parts of y.
struct Space {
  size_t rows, part, total;
};
Space space_of(const MoeArgs& a, const DeviceCaps& caps) {
  Space s;
  s.rows = up256(sizeof(Reached));
  s.part = s.rows + up256((size_t)a.T * a.top * kMoeParts * mx_pitch(a.F) * 2);
  const int slices = down_slices(a, caps);
  s.total = s.part + (slices > 1 ? up256((size_t)slices * a.T * a.H * 4) : 0);
  return s;
}

template <typename K>
hipError_t allow_lds(K k, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int DT, int COLS>
hipError_t up(const MoeArgs& a, const DeviceCaps& caps, char* ws, const Space& sp, hipStream_t st) {
  const int64_t Fp = mx_pitch(a.F);
  const int64_t items = std::min<int64_t>(a.E, a.T * a.top) * (Fp / 16);
  constexpr int lds = NW * (kSlots * kSlot + column_bytes(mx_parts(DT), COLS));
  constexpr int fixed = sizeof(Routing) + 2 * NW * RT * 16 * (COLS + 1) * 4;
  const int64_t per_cu = lds + fixed <= 80 * 1024 ? 2 : 1;
  const int64_t wgs = std::max<int64_t>(1, std::min<int64_t>(items, per_cu * caps.cus));
  const hipError_t e = allow_lds(moe_up_kernel<DT, COLS>, lds);
  if (e != hipSuccess) return e;
  moe_up_kernel<DT, COLS><<<(unsigned)wgs, NW * 64, lds, st>>>(
      a.x, (int)a.ldx, (int)a.Hx, a.logits, a.ldt, a.ldl, a.W1, a.w1_scales, (int)a.T, (int)a.E, a.top, a.renorm,
      (int)mx_pitch(a.H), (int)a.F, (int)Fp, reinterpret_cast<uint16_t*>(ws + sp.rows), reinterpret_cast<Reached*>(ws));
  return hipGetLastError();
}

template <int DT, int COLS, int SLOTS, int WAVES>
hipError_t down(const MoeArgs& a, char* ws, const Space& sp, int S, hipStream_t st) {
  const int lds = down_lds(a, COLS, SLOTS, WAVES);
  const hipError_t e = allow_lds(moe_down_kernel<DT, COLS, SLOTS, WAVES>, lds);
  if (e != hipSuccess) return e;
  const int groups = (int)((a.H + RT * 16 - 1) / (RT * 16));
  moe_down_kernel<DT, COLS, SLOTS, WAVES><<<(unsigned)(groups * S), WAVES * 64, lds, st>>>(
      reinterpret_cast<const uint16_t*>(ws + sp.rows), reinterpret_cast<const Reached*>(ws), a.W2, a.w2_scales, (int)a.T,
      (int)a.E, a.top, (int)a.H, (int)mx_pitch(a.F), S, a.out, a.ldo, S > 1 ? reinterpret_cast<float*>(ws + sp.part) : nullptr);
  return hipGetLastError();
}

// Whether the second launch takes four tokens at a time: to four tokens an expert on average (three parts of
// sixteen columns are more to fetch than those of the first launch: 13 tokens, 2 of 8 experts of 4096 x 11008,
// 134 us in all instead of 160 with sixteen; 16 tokens 164 and 166, 24 tokens 191 and 180), and as long as
// the columns that it keeps in LDS leave place for two workgroups a CU, up to 36 tokens (48 tokens, 8 of 128
// experts of 2048 x 768, 119 us, 105 with sixteen columns, from registers).
bool few_down(const MoeArgs& a) { return (few_each(a) || a.T * a.top <= 4 * a.E) && down_lds(a, 4, 2, NW) <= 80 * 1024; }

// Rings of three units where two workgroups of them share a CU, else of two (the sums of many tokens
// take the place; of eight waves with a CU to themselves, three are slower: 20.2 us instead of 19.9 for
// one token and 8 of 128 experts).
template <int DT, int COLS>
hipError_t down_ring(const MoeArgs& a, char* ws, const Space& sp, int S, hipStream_t st) {
  return down_lds(a, COLS, 3, NW) <= 80 * 1024 ? down<DT, COLS, 3, NW>(a, ws, sp, S, st) : down<DT, COLS, 2, NW>(a, ws, sp, S, st);
}

template <int DT>
hipError_t both(const MoeArgs& a, const DeviceCaps& caps, char* ws, const Space& sp, int S, hipStream_t st) {
  const hipError_t e = few_each(a) ? up<DT, 4>(a, caps, ws, sp, st) : up<DT, 16>(a, caps, ws, sp, st);
  if (e != hipSuccess) return e;
  if (down_alone(a, caps)) return down<DT, 4, 2, 8>(a, ws, sp, S, st);
  return few_down(a) ? down_ring<DT, 4>(a, ws, sp, S, st) : down_ring<DT, 16>(a, ws, sp, S, st);
}

template <int DT>
hipError_t run(const MoeArgs& a, const DeviceCaps& caps, char* ws, hipStream_t st) {
  const Space sp = space_of(a, caps);
  const int S = down_slices(a, caps);
  const hipError_t e = both<DT>(a, caps, ws, sp, S, st);
  if (e != hipSuccess || S == 1) return e;
  moe_join_kernel<DT><<<dim3((unsigned)((a.H + 255) / 256), (unsigned)a.T), 256, 0, st>>>(
      reinterpret_cast<const float*>(ws + sp.part), reinterpret_cast<const Reached*>(ws), (int)a.T, (int)a.H, S, a.out, a.ldo);
  return hipGetLastError();
}

}  // namespace

size_t moe_workspace_bytes(const MoeArgs& a, const DeviceCaps& caps) { return space_of(a, caps).total; }

hipError_t launch_moe(const MoeArgs& a, const DeviceCaps& caps, void* ws, hipStream_t st) {
  char* w = static_cast<char*>(ws);
  switch (a.dt) {
    case W4_DT_F32: return run<W4_DT_F32>(a, caps, w, st);
    case W4_DT_F16: return run<W4_DT_F16>(a, caps, w, st);
    default: return run<W4_DT_BF16>(a, caps, w, st);
  }
}

}  // namespace w4
