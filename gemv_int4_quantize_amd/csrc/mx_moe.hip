// A mixture-of-experts layer on microscaled 4-bit weights for a few tokens (mx4_moe), for gfx950.
// For token t with logits z over E experts, j over the `top` largest (by value, then lower index):
//   g_j = exp(z_j - max z) / total,  total over the chosen (renormalized) or over all experts
//   a_j = silu(W1g[j] x) * (W1u[j] x),  y = sum_j g_j W2[j] a_j
// in two launches: the choice of experts and g_j a_j, then the sum over experts (and, where the
// rows of y alone would leave compute units idle, a third that adds its parts).
//
// What bounds it: the weights of the experts that some token reaches, each read once.  They go from
// memory straight to registers, are widened to bf16 (exactly: two significant bits) and multiplied on
// the matrix cores with up to sixteen tokens as the columns.  The activations enter as bf16 parts
// whose sum they are (one of bf16, two of fp16, three of fp32), and so does g_j a_j (two parts,
// 16 bits; three for fp32): the matrix cores have time for it, and what lies between the two
// products is not rounded to bf16's eight bits.
#include <algorithm>

#include "api_common.h"
#include "launch.h"
#include "mx.h"

namespace w4 {

namespace {

constexpr int kNonTemporal = 2;  // cache-policy operand of a buffer load
constexpr int kTokens = kMoeTokens, kMaxTop = kMoeTop, kMaxExperts = kMoeExperts;
constexpr int kNone = 0x7FFF0000;  // a buffer offset that is out of range: 0 without a request
constexpr uint32_t kOverflows = 253;  // stored exponents from which on a value may pass bf16's range
constexpr int NW = 8;              // waves of a workgroup

// The experts that the tokens reach, in the order of their numbers, as the second launch takes them
// from the workspace: expert, bit set of its tokens, and its first row of a_j (rows in token order).
struct Reached {
  uint64_t bad;  // tokens whose logits hold a NaN or +infinity
  int count;
  int expert[kMaxExperts];
  int first[kMaxExperts];
  uint64_t tokens[kMaxExperts];
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s, 64);
  return v;
}

template <int DT>
__device__ __forceinline__ float logit(const void* z, int64_t i) {
  return elem_to_f32<DT>(static_cast<const typename Elem<DT>::type*>(z)[i]);
}

struct Routing {
  uint64_t tokens[kMaxExperts];  // of each expert
  uint64_t bad;
  int count;
  int expert[kMaxExperts], first[kMaxExperts];  // those reached
  short chosen[kTokens][kMaxTop];
  float weight[kTokens][kMaxTop];
};

// Values as unsigned integers of the same order.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Every workgroup makes the choice for all tokens, a wave a token: 64 lanes hold E / 64 logits each and
// take the largest out `top` times.
template <int DT>
__device__ __forceinline__ void route(Routing& s, const void* __restrict__ logits, int64_t ldl, int T, int E, int top,
                                      bool renorm) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int C = kMaxExperts / 64;
  for (int e = tid; e < E; e += NW * 64) s.tokens[e] = 0;
  if (tid == 0) s.bad = 0;
  __syncthreads();
  const uint32_t masked = order_key(-__builtin_inff());
  for (int t = wave; t < T; t += NW) {
    uint32_t key[C];
    float v[C];
    bool odd = false;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = c * 64 + lane;
      v[c] = e < E ? logit<DT>(logits, t * ldl + e) : -__builtin_inff();
      odd |= !(v[c] < __builtin_inff());
      // -0 and +0 are equal
      key[c] = e < E ? order_key(v[c] + 0.0f) : 0u;
    }
    if (__ballot(odd) != 0) {
      if (lane == 0) atomicOr(reinterpret_cast<unsigned long long*>(&s.bad), 1ull << t);
      if (lane < top) s.chosen[t][lane] = -1;
      continue;
    }
    float mx = 0.0f, total = 0.0f;
    for (int j = 0; j < top; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) best = umax(best, key[c]);
      best = wave_umax(best);
      int expert = -1;
      float w = 0.0f;
      if (best > masked) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint64_t at = __ballot(key[c] == best);
          if (expert < 0 && at != 0) {
            const int l = __builtin_ctzll(at);
            expert = c * 64 + l;
            if (lane == l) key[c] = 0;
          }
        }
        const float z = __uint_as_float(best & 0x80000000u ? best & 0x7FFFFFFFu : ~best);
        if (j == 0) mx = z;
        w = expf(z - mx);
        total += w;
      }
      if (lane == 0) {
        s.chosen[t][j] = (short)expert;
        s.weight[t][j] = w;
        if (expert >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&s.tokens[expert]), 1ull << t);
      }
    }
    __builtin_amdgcn_wave_barrier();  // lane 0's writes, then the other lanes' reads
    if (!renorm) {
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) sum += expf(v[c] - mx);
      total = wave_sum(sum);
    }
    if (lane < top) s.weight[t][lane] = s.weight[t][lane] / total;
  }
  __syncthreads();
  if (wave == 0) {
    int count = 0, rows = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const uint64_t m = e < E ? s.tokens[e] : 0;
      const uint64_t live = __ballot(m != 0);
      int n = __popcll(m), before = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(before, d, 64);
        if (lane >= d) before += up;
      }
      if (m != 0) {
        const int at = count + __popcll(live & ((1ull << lane) - 1));
        s.expert[at] = e;
        s.first[at] = rows + before - n;
      }
      count += __popcll(live);
      rows += __shfl(before, 63, 64);
    }
    if (lane == 0) s.count = count;
  }
  __syncthreads();
}

// The i-th set bit of m.
__device__ __forceinline__ int nth_bit(uint64_t m, int i) {
  for (int k = 0; k < i; ++k) m &= m - 1;
  return __builtin_ctzll(m);
}

template <int AUX>
__device__ __forceinline__ u32x4 load16(rsrc_t r, int off, int soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, AUX));
}
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A wave's RT tiles of 16 weight rows over a unit of 256 columns: lane l takes two blocks of 32 columns
// (from 64 (l / 16)) of row l % 16, so that its loads touch whole 128-byte lines, and the same
// columns of the token that column l % 16 stands for.
template <int RT>
struct Unit {
  u32x4 w[RT][2];
  uint32_t e[RT];
};

// Tiles [r0, r0 + n) from weight rows [first, first + rows) (rows past them: 0).
template <int RT>
__device__ __forceinline__ void load_tiles(Unit<RT>& t, int r0, int n, const uint8_t* W, const uint8_t* we, size_t first,
                                           uint32_t rows, int P, int u, int lane) {
  const int row = P >> 1, erow = P >> 5, r16 = lane & 15, q4 = lane >> 4;
  const rsrc_t rw = mx_rsrc(W + first * row, rows * (uint32_t)row);
  const rsrc_t re = mx_rsrc(we + first * erow, rows * (uint32_t)erow);
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (r < r0 || r >= r0 + n) continue;
    const int at = (r - r0) * 16 + r16;
#pragma unroll
    for (int h = 0; h < 2; ++h) t.w[r][h] = load16<kNonTemporal>(rw, at * row + q4 * 32 + h * 16, u * 128);
    t.e[r] = __builtin_amdgcn_raw_buffer_load_b16(re, at * erow + q4 * 2, u * 8, 0);
  }
}

// acc[r][b] += tile r times the sixteen columns of block b, whose parts (`step` bytes after one another)
// begin at xo[b].  in: the lane's 64 columns lie in the row (else they are the next row's).
template <int RT, int NP, int NB>
__device__ __forceinline__ void multiply(const Unit<RT>& t, bool in, rsrc_t rx, const int (&xo)[NB], uint32_t blocks, int step,
                                         f32x4 (&acc)[RT][NB]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float p[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) p[r] = in ? mx_power((t.e[r] >> (8 * h)) & 255u) : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 a[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) a[r] = mx_bf16x8(in ? t.w[r][h][i] : 0u, p[r]);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (NB > 1 && (blocks >> b & 1) == 0) continue;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const u32x4 x = load16<0>(rx, xo[b] + h * 64 + i * 16, k * step);
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[r][b] = mfma16(a[r], x, acc[r][b]);
        }
      }
    }
  }
}

// The waves' sums of block b in LDS.
template <int RT, int NB>
__device__ __forceinline__ void put_sums(float (*sums)[RT * 16][17], const f32x4 (&acc)[RT][NB], int b, int wave, int lane) {
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[wave][r * 16 + (lane >> 4) * 4 + i][lane & 15] = acc[r][b][i];
}

// First launch: the choice, then items of R x 16 gate rows and the same up rows of one expert, whose
// contraction the workgroup's waves share.  x [T][NP][ldx] bf16 parts, Hx (a multiple of 64) columns
// of each to read; a [rows][HP][Fp] bf16 parts of g_j a_j, a row for each expert and token of it.
template <int DT, int LDT, int R, int NB>
__global__ __launch_bounds__(NW * 64) void moe_up_kernel(const uint16_t* __restrict__ x, int ldx, int Hx,
                                                         const void* __restrict__ logits, int64_t ldl,
                                                         const uint8_t* __restrict__ W, const uint8_t* __restrict__ we, int T,
                                                         int E, int top, int renorm, int P, int F, int Fp,
                                                         uint16_t* __restrict__ a, Reached* __restrict__ reached) {
  constexpr int NP = mx_parts(DT), HP = moe_parts(DT), RT = 2 * R;
  __shared__ Routing s;
  __shared__ float sums[NW][RT * 16][17];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  route<LDT>(s, logits, ldl, T, E, top, renorm != 0);
  if (blockIdx.x == 0) {  // for the second launch
    for (int i = tid; i < s.count; i += NW * 64) {
      reached->expert[i] = s.expert[i];
      reached->first[i] = s.first[i];
      reached->tokens[i] = s.tokens[s.expert[i]];
    }
    if (tid == 0) {
      reached->count = s.count;
      reached->bad = s.bad;
    }
  }
  const int tiles = Fp / (16 * R), items = s.count * tiles;
  const int units = (P + 255) >> 8, per = (units + NW - 1) / NW;
  const int u0 = min(wave * per, units), u1 = min(u0 + per, units);
  const int r16 = lane & 15, q4 = lane >> 4;
  const rsrc_t rx = mx_rsrc(x, (uint32_t)T * (uint32_t)(NP * ldx) * 2u);
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int slot = item / tiles, f0 = (item - slot * tiles) * 16 * R;
    const int e = __builtin_amdgcn_readfirstlane(s.expert[slot]);
    const uint64_t tokens = s.tokens[e];
    const int cols = __popcll(tokens);
    const uint32_t rows = (uint32_t)max(0, min(16 * R, F - f0));
    int tok[NB];
    uint32_t blocks = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      tok[b] = b * 16 + r16 < cols ? nth_bit(tokens, b * 16 + r16) * (NP * ldx * 2) : kNone;
      blocks |= (b * 16 < cols ? 1u : 0u) << b;
    }
    blocks = __builtin_amdgcn_readfirstlane(blocks);
    f32x4 acc[RT][NB];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[r][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int u = u0; u < u1; ++u) {
      Unit<RT> t;
      load_tiles<RT>(t, 0, R, W, we, (size_t)e * 2 * F + f0, rows, P, u, lane);
      load_tiles<RT>(t, R, R, W, we, ((size_t)e * 2 + 1) * F + f0, rows, P, u, lane);
      const int col = u * 256 + q4 * 64;
      int xo[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) xo[b] = col < Hx && tok[b] != kNone ? tok[b] + col * 2 : kNone;
      multiply<RT, NP, NB>(t, col < P, rx, xo, blocks, ldx * 2, acc);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (NB > 1 && (blocks >> b & 1) == 0) break;
      put_sums<RT, NB>(sums, acc, b, wave, lane);
      __syncthreads();
      for (int i = tid; i < 16 * R * 16; i += NW * 64) {
        const int f = i % (16 * R), c = i / (16 * R), col = b * 16 + c;
        if (col >= cols) break;  // columns ascend with i
        float g = 0.0f, up = 0.0f;
#pragma unroll
        for (int v = 0; v < NW; ++v) {
          g += sums[v][f][c];
          up += sums[v][16 * R + f][c];
        }
        const int t = nth_bit(tokens, col);
        float w = 0.0f;
        for (int j = 0; j < top; ++j) w = s.chosen[t][j] == e ? s.weight[t][j] : w;
        float v = g / (1.0f + expf(-g)) * up * w;
        uint16_t* o = a + (size_t)(s.first[slot] + col) * (HP * Fp) + f0 + f;
        // parts as of mx_parts_kernel: the rest cut to eight bits
        const bool odd = (__float_as_uint(v) & 0x7FFFFFFFu) >= 0x7F800000u;
#pragma unroll
        for (int k = 0; k < HP; ++k) {
          uint32_t bits = __float_as_uint(v) >> 16;
          if (k == HP - 1 && !odd) bits = pack_bf16x2(v, 0.0f) & 0xFFFFu;  // the last one rounded
          if (odd) bits = k > 0 ? 0u : (__float_as_uint(v) & 0x7FFFFFu) != 0 ? 0x7FC0u : bits;
          o[(size_t)k * Fp] = (uint16_t)bits;
          v -= __uint_as_float(bits << 16);
          if (odd) v = 0.0f;
        }
      }
      __syncthreads();
    }
  }
}

template <int DT>
__device__ __forceinline__ void store(void* out, int64_t i, float v) {
  if constexpr (DT == W4_DT_F32) static_cast<float*>(out)[i] = v;
  else if constexpr (DT == W4_DT_BF16) static_cast<uint16_t*>(out)[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
  else static_cast<uint16_t*>(out)[i] = f32_to_f16_bits(v);
}

// Second launch: RT x 16 rows of y for a workgroup, whose waves share the units of all reached experts,
// with those of the other S - 1 workgroups of these rows.  The columns are the tokens, those that an
// expert does not have being 0, so that the sum over experts stays in registers.
template <int DT, int RT, int NB>
__global__ __launch_bounds__(NW * 64) void moe_down_kernel(const uint16_t* __restrict__ a, const Reached* __restrict__ reached,
                                                           const uint8_t* __restrict__ W, const uint8_t* __restrict__ we, int T,
                                                           int rows_a, int H, int Fp, int S, void* __restrict__ out, int64_t ldo,
                                                           float* __restrict__ part) {
  constexpr int HP = moe_parts(DT);
  __shared__ Reached s;
  __shared__ float sums[NW][RT * 16][17];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int count = __builtin_amdgcn_readfirstlane(reached->count);
  const uint64_t bad = reached->bad;
  for (int i = tid; i < count; i += NW * 64) {
    s.expert[i] = reached->expert[i];
    s.first[i] = reached->first[i];
    s.tokens[i] = reached->tokens[i];
  }
  __syncthreads();
  const int group = blockIdx.x / (unsigned)S, slice = blockIdx.x - group * S;
  const int h0 = group * 16 * RT;
  const uint32_t rows = (uint32_t)min(16 * RT, H - h0);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int of_expert = (Fp + 255) >> 8, units = count * of_expert;
  const int per = (units + S * NW - 1) / (S * NW);
  const int u0 = min((slice * NW + wave) * per, units), u1 = min(u0 + per, units);
  const rsrc_t rx = mx_rsrc(a, (uint32_t)rows_a * (uint32_t)(HP * Fp) * 2u);
  f32x4 acc[RT][NB];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[r][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = u0; i < u1; ++i) {
    const int slot = i / of_expert, u = i - slot * of_expert;
    const int e = __builtin_amdgcn_readfirstlane(s.expert[slot]);
    Unit<RT> t;
    load_tiles<RT>(t, 0, RT, W, we, (size_t)e * H + h0, rows, Fp, u, lane);
    const uint64_t tokens = s.tokens[slot];
    const int col = u * 256 + q4 * 64;
    int xo[NB];
    bool has[NB];
    uint32_t blocks = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int tk = b * 16 + r16;
      has[b] = (tokens >> tk & 1) != 0;
      const int at = s.first[slot] + __popcll(tokens & ((1ull << tk) - 1));
      xo[b] = has[b] && col < Fp ? (at * (HP * Fp) + col) * 2 : kNone;
      blocks |= ((tokens >> (b * 16) & 0xFFFF) != 0 ? 1u : 0u) << b;
    }
    blocks = __builtin_amdgcn_readfirstlane(blocks);
    // a weight that is NaN or past bf16's range must not reach the tokens without the expert, whose
    // columns are 0: theirs are put back, a tile at a time
    bool odd = false;
#pragma unroll
    for (int r = 0; r < RT; ++r) odd |= (t.e[r] & 255u) >= kOverflows || (t.e[r] >> 8) >= kOverflows;
    if (__ballot(odd) == 0) {
      multiply<RT, HP, NB>(t, col < Fp, rx, xo, blocks, Fp * 2, acc);
    } else {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const Unit<1> one = {{{t.w[r][0], t.w[r][1]}}, {t.e[r]}};
        f32x4 sum[1][NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) sum[0][b] = acc[r][b];
        multiply<1, HP, NB>(one, col < Fp, rx, xo, blocks, Fp * 2, sum);
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[r][b] = has[b] ? sum[0][b] : acc[r][b];
      }
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (b * 16 >= T) break;
    put_sums<RT, NB>(sums, acc, b, wave, lane);
    __syncthreads();
    for (int i = tid; i < RT * 16 * 16; i += NW * 64) {
      const int h = i % (RT * 16), c = i / (RT * 16), t = b * 16 + c;
      if (t >= T) break;
      if (h >= (int)rows) continue;
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < NW; ++k) v += sums[k][h][c];
      if (part != nullptr) part[((size_t)slice * T + t) * H + h0 + h] = v;
      else store<DT>(out, t * ldo + h0 + h, (bad >> t & 1) != 0 ? __builtin_nanf("") : v);
    }
    __syncthreads();
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

// Rows of the second launch's workgroups, and workgroups for the same rows: about two a CU.
constexpr int kDownTiles = 4;
int down_slices(const MoeArgs& a, const DeviceCaps& caps) {
  const int64_t groups = (a.H + kDownTiles * 16 - 1) / (kDownTiles * 16);
  const int64_t units = std::min<int64_t>(a.E, a.T * a.top) * ((mx_pitch(a.F) + 255) / 256);
  int64_t s = (2 * (int64_t)caps.cus + groups - 1) / groups;
  s = std::min(s, (units + NW - 1) / NW);
  return (int)std::max<int64_t>(1, std::min<int64_t>(s, 16));
}

// The workspace: what the experts reached are, g_j a_j, parts of y.
struct Space {
  size_t rows, part, total;
};
Space space_of(const MoeArgs& a, const DeviceCaps& caps) {
  Space s;
  s.rows = up256(sizeof(Reached));
  s.part = s.rows + up256((size_t)a.T * a.top * moe_parts(a.dt) * mx_pitch(a.F) * 2);
  const int slices = down_slices(a, caps);
  s.total = s.part + (slices > 1 ? up256((size_t)slices * a.T * a.H * 4) : 0);
  return s;
}

template <int DT, int LDT, int R, int NB>
hipError_t up(const MoeArgs& a, const DeviceCaps& caps, char* ws, const Space& sp, hipStream_t st) {
  const int64_t Fp = mx_pitch(a.F);
  const int64_t items = std::min<int64_t>(a.E, a.T * a.top) * (Fp / (16 * R));
  const int64_t wgs = std::max<int64_t>(1, std::min<int64_t>(items, 2 * (int64_t)caps.cus));
  moe_up_kernel<DT, LDT, R, NB><<<(unsigned)wgs, NW * 64, 0, st>>>(
      a.x, (int)a.ldx, (int)a.Hx, a.logits, a.ldl, a.W1, a.w1_scales, (int)a.T, (int)a.E, a.top, a.renorm, (int)mx_pitch(a.H),
      (int)a.F, (int)Fp, reinterpret_cast<uint16_t*>(ws + sp.rows), reinterpret_cast<Reached*>(ws));
  return hipGetLastError();
}

template <int DT, int LDT>
hipError_t run_up(const MoeArgs& a, const DeviceCaps& caps, char* ws, const Space& sp, hipStream_t st) {
  const int64_t items = std::min<int64_t>(a.E, a.T * a.top) * (mx_pitch(a.F) / 32);
  const bool few = items < 2 * (int64_t)caps.cus;
  if (a.T <= 16) return few ? up<DT, LDT, 1, 1>(a, caps, ws, sp, st) : up<DT, LDT, 2, 1>(a, caps, ws, sp, st);
  return up<DT, LDT, 2, 4>(a, caps, ws, sp, st);
}

template <int DT>
hipError_t run(const MoeArgs& a, const DeviceCaps& caps, char* ws, hipStream_t st) {
  const Space sp = space_of(a, caps);
  hipError_t e;
  if (a.ldt == W4_DT_F32) e = run_up<DT, W4_DT_F32>(a, caps, ws, sp, st);
  else if (a.ldt == W4_DT_F16) e = run_up<DT, W4_DT_F16>(a, caps, ws, sp, st);
  else e = run_up<DT, W4_DT_BF16>(a, caps, ws, sp, st);
  if (e != hipSuccess) return e;
  const int S = down_slices(a, caps);
  const Reached* reached = reinterpret_cast<const Reached*>(ws);
  const uint16_t* rows = reinterpret_cast<const uint16_t*>(ws + sp.rows);
  float* part = S > 1 ? reinterpret_cast<float*>(ws + sp.part) : nullptr;
  const int groups = (int)((a.H + kDownTiles * 16 - 1) / (kDownTiles * 16));
  auto k = a.T <= 16 ? moe_down_kernel<DT, kDownTiles, 1> : moe_down_kernel<DT, kDownTiles, 4>;
  k<<<(unsigned)(groups * S), NW * 64, 0, st>>>(rows, reached, a.W2, a.w2_scales, (int)a.T, (int)(a.T * a.top), (int)a.H,
                                                (int)mx_pitch(a.F), S, a.out, a.ldo, part);
  e = hipGetLastError();
  if (e != hipSuccess || S == 1) return e;
  moe_join_kernel<DT><<<dim3((unsigned)((a.H + 255) / 256), (unsigned)a.T), 256, 0, st>>>(part, reached, (int)a.T, (int)a.H, S,
                                                                                        a.out, a.ldo);
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
