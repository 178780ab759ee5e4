// Scores of given tokens (tok_logprobs) and their gradient, for gfx950.  For a row z of V
// logits, mx = max z, d = (z - mx) / T:
//   S = sum e^d,  logprob = d_t - log S,  entropy = log S - sum e^d d / S.
// The maximum is taken off before the division by T, so that nothing overflows (a mask of
// the type's lowest value divided by a small T) and the most likely tokens keep their bits.
//
// Forward: one pass over the logits.  Each thread keeps the maximum of what it has read and
// S and sum e^d d relative to it, rescaled once per group of kU chunks (a group's maximum
// is taken before its exponentials, so the rescaling costs one exponential per group and
// not one per new maximum).  A row is read by one workgroup, or cut into parts whose
// results a second, one-wave launch joins, when there are few rows.
//
// Alternatives: the maxima of 128 pairs of threads are on hand after the pass, and the k-th
// largest of them is a threshold that at least k logits reach.  Each thread has also kept the
// maximum of each of (up to) 16 runs of its chunks, so that only the few runs that reach the
// threshold are read again; what reaches it in them is ranked by counting.  (Reading all of
// the pairs' chunks again cost 17 us of 112 at M = 2048, V = 128256 bf16.)  Rows with too many
// logits at the threshold (many equal ones, or fewer unmasked than alternatives) collect
// those above it, and of those equal to it the lowest ids in order, from the pairs' chunks.
//
// Measured at M = 2048, V = 128256 bf16: forward without alternatives 95-100 us (5.3-5.5 TB/s),
// with five 104 (5.0 TB/s), gradient 205 us (5.1 TB/s of reads and writes; stores that bypass the
// caches, 319 -> 302 us for the pair).  The forward pass is bound by the vector units and by memory
// together: counters have the former busy 77% of the cycles (74% with alternatives) while a plain
// read reaches 6.75 TB/s; the gradient by memory (vector units 31%).  Four fp32 rows with twenty
// alternatives: 10 us and 5 for the join, both mostly latency.
#include <algorithm>

#include "api_common.h"
#include "launch.h"
#include "rows.h"

namespace w4 {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.4028234663852886e38f;
// e^d d is 0 below this (exp2 is): arguments are held above it, so that -infinity gives 0
// and not infinity * 0
constexpr float kFloor = -1.0e4f;

constexpr int kT = 256;       // threads
constexpr int kPairs = kT / 2;
constexpr int kRuns = 16;     // runs of a thread's chunks whose maxima are kept
constexpr int kMaxTop = 64;
constexpr int kCand = 1024;   // logits above the threshold that are held at a time
constexpr int kMaxParts = 64; // parts of a row, one per lane of the joining wave
constexpr int kMinSeg = kT * 32;  // measured against 8 and 16 a thread: 16 rows, top 20, 19.4 -> 16.4 us

// Running softmax statistics: the largest logit, S and sum e^d d (in units of log2) relative
// to it.  m is -infinity while only masked logits were seen.
struct Stat {
  float m, s, t;
};

// The statistics of both, relative to the larger maximum.
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float c) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  const float base = fmaxf(r.m, kLowest);
  // an infinite distance scales a zero sum by zero
  const float da = fminf((base - fmaxf(a.m, kLowest)) * c, 1e30f), db = fminf((base - fmaxf(b.m, kLowest)) * c, 1e30f);
  const float ea = __builtin_amdgcn_exp2f(-da), eb = __builtin_amdgcn_exp2f(-db);
  r.s = a.s * ea + b.s * eb;
  r.t = (a.t - da * a.s) * ea + (b.t - db * b.s) * eb;
  return r;
}

__device__ __forceinline__ Stat wave_join(Stat st, float c) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const Stat p = {__shfl_xor(st.m, o), __shfl_xor(st.s, o), __shfl_xor(st.t, o)};
    st = join(st, p, c);
  }
  return st;
}

// One group of N logits into the running statistics; their maximum is joined to `run`.
template <int N>
__device__ __forceinline__ void take(Stat& st, const float (&v)[N], float c, float& run) {
  float m = v[0];
#pragma unroll
  for (int j = 1; j < N; j += 2) m = __builtin_fmaxf(__builtin_fmaxf(m, v[j]), v[j + 1 < N ? j + 1 : j]);
  run = __builtin_fmaxf(run, m);
  m = __builtin_fmaxf(m, st.m);
  const float base = __builtin_fmaxf(m, kLowest);
  const float d = __builtin_fminf((base - __builtin_fmaxf(st.m, kLowest)) * c, 1e30f);
  const float e = __builtin_amdgcn_exp2f(-d);
  float s = st.s * e, t = (st.t - d * st.s) * e;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float x = (v[j] - base) * c;
    const float p = __builtin_amdgcn_exp2f(x);
    s += p;
    t = __builtin_fmaf(p, __builtin_fmaxf(x, kFloor), t);
  }
  st.m = m;
  st.s = s;
  st.t = t;
}

// What a row's statistics say.  A NaN or +infinity among the logits makes S NaN (infinity -
// infinity); nothing but -infinity leaves S at 0.
struct RowOut {
  float mx, logs, ent;
  bool bad, empty;
};
__device__ __forceinline__ RowOut row_out(const Stat& st) {
  RowOut r;
  r.bad = !(st.s == st.s) || st.m == INFINITY;
  r.empty = !r.bad && st.m == -INFINITY;
  r.mx = st.m;
  r.logs = r.empty ? 0.0f : logf(st.s);
  r.ent = r.empty ? 0.0f : r.logs - st.t / st.s * kLn2;
  if (r.bad) r.mx = r.logs = r.ent = __uint_as_float(0x7FC00000u);
  return r;
}
__device__ __forceinline__ float row_logprob(const RowOut& r, float z, float inv_t) {
  return r.bad ? r.mx : r.empty ? -INFINITY : (z - r.mx) * inv_t - r.logs;
}

// Largest first, then the lower id.
__device__ __forceinline__ bool before(float va, int ja, float vb, int jb) { return va > vb || (va == vb && ja < jb); }

// A row's target and its logit, read early: the two loads depend on one another.
struct Target {
  int64_t t;
  float z;
};
template <int DT>
__device__ __forceinline__ Target load_target(const TokArgs& a, int64_t row) {
  typedef typename Elem<DT>::type E;
  Target r;
  r.t = a.targets[row];
  const bool in = r.t >= 0 && r.t < a.V;
  r.z = elem_to_f32<DT>((static_cast<const E*>(a.z) + row * a.ld)[in ? r.t : 0]);
  return r;
}

__device__ __forceinline__ void write_row(const TokArgs& a, int64_t row, const RowOut& r, const Target& t) {
  a.ent[row] = r.ent;
  a.stats[2 * row] = r.mx;
  a.stats[2 * row + 1] = r.logs;
  const float nan = __uint_as_float(0x7FC00000u);
  a.lp[row] = t.t == a.ignore ? 0.0f : t.t < 0 || t.t >= a.V ? nan : row_logprob(r, t.z, a.inv_t);
}

// One part of a row's results, for the joining launch: statistics, then `top` (logit, id)
// pairs in order.
struct Part {
  Stat st;
  float pad;
};

// A float's upper half, rounded towards +infinity: not below the float, and the float itself
// for bf16 values.
__device__ __forceinline__ uint16_t up16(float v) {
  const uint32_t u = __float_as_uint(v);
  return (uint16_t)((u + (u >> 31 ? 0u : 0xFFFFu)) >> 16);
}

struct __attribute__((aligned(16))) TopShared {
  float gm[kPairs];
  float cv[kCand];  // logits above the threshold and their ids; then the result
  int cj[kCand];
  float tau;
  int ng;                // logits above the threshold that were seen
  int nl;                // entries of runs
  uint16_t runs[kT];     // runs to read again: run * kT + thread
  uint8_t list[kPairs];  // pairs whose maximum reaches the threshold, in order
  int tie[kMaxTop];
  int wsum[kT / 64];
};

// The k-th largest (equal values count each) of the n values in v, by counting, to sh.tau;
// n is a multiple of 4.  All threads call it.
__device__ __forceinline__ void kth_largest(const float* v, int n, int k, TopShared& sh) {
  const f32x4* v4 = reinterpret_cast<const f32x4*>(v);
  for (int i = threadIdx.x; i < n; i += kT) {
    const float x = v[i];
    int above = 0, equal = 0;
#pragma unroll 4
    for (int j = 0; j < n / 4; ++j) {
      const f32x4 o = v4[j];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        above += o[u] > x ? 1 : 0;
        equal += o[u] == x ? 1 : 0;
      }
    }
    if (above < k && above + equal >= k) sh.tau = x;  // every such thread writes the same value
  }
}

// The same of the kPairs pair maxima, to sh.tau.  For small k one wave takes the largest off
// until k are gone: less work in all than counting, which tells where every workgroup of a CU
// does this at about the same time.  Larger k count, two threads a value: 20 rounds of the
// former took 4 us of a launch for few rows.
__device__ __forceinline__ void kth_pair(int k, TopShared& sh) {
  const int tid = threadIdx.x;
  if (k > 8) {
    const float x = sh.gm[tid >> 1];
    const f32x4* v4 = reinterpret_cast<const f32x4*>(sh.gm) + (tid & 1) * (kPairs / 8);
    int n = 0;  // values above x, and equal ones in the upper half
#pragma unroll
    for (int j = 0; j < kPairs / 8; ++j) {
      const f32x4 o = v4[j];
#pragma unroll
      for (int u = 0; u < 4; ++u) n += o[u] > x ? 1 : o[u] == x ? 0x10000 : 0;
    }
    n += __shfl_xor(n, 1);
    const int above = n & 0xFFFF;
    if (above < k && above + (n >> 16) >= k) sh.tau = x;
    return;
  }
  if (tid >= 64) return;
  const float nan = __uint_as_float(0x7FC00000u);
  float a = sh.gm[tid], b = sh.gm[tid + 64];
  for (;;) {
    const float m = wave_max(__builtin_fmaxf(__builtin_fmaxf(a, b), -INFINITY));
    k -= __popcll(__ballot(a == m)) + __popcll(__ballot(b == m));
    if (k <= 0) {
      if (tid == 0) sh.tau = m;
      return;
    }
    a = a == m ? nan : a;
    b = b == m ? nan : b;
  }
}

// The `top` best of the ng (<= kCand) pairs in sh.cv / sh.cj, in order, to their front: ranked by
// counting, in any order (the last group of four is filled up with pairs that come after
// every other).  Entries past ng are left to the caller.
__device__ __forceinline__ void rank_top(int ng, int top, TopShared& sh) {
  const int tid = threadIdx.x;
  if (tid < 3 && ng + tid < kCand) {
    sh.cv[ng + tid] = -INFINITY;
    sh.cj[ng + tid] = 0x7FFFFFFF;
  }
  __syncthreads();
  float v[kCand / kT];
  int j[kCand / kT], rank[kCand / kT];
#pragma unroll
  for (int q = 0; q < kCand / kT; ++q) {
    const int i = tid + q * kT;
    rank[q] = kMaxTop;
    if (i < ng) {
      v[q] = sh.cv[i];
      j[q] = sh.cj[i];
      int r = 0;
#pragma unroll 2
      for (int o = 0; o < (ng + 3) / 4; ++o) {
        const f32x4 ov = reinterpret_cast<const f32x4*>(sh.cv)[o];
        const u32x4 oj = reinterpret_cast<const u32x4*>(sh.cj)[o];
#pragma unroll
        for (int u = 0; u < 4; ++u) r += before(ov[u], (int)oj[u], v[q], j[q]) ? 1 : 0;
      }
      rank[q] = r;
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kCand / kT; ++q)
    if (rank[q] < top) {
      sh.cv[rank[q]] = v[q];
      sh.cj[rank[q]] = j[q];
    }
}

// The `top` best (logit, id) pairs of the n logits from z, in order, to sh.cv / sh.cj [top]
// (ids from z; past n: -infinity and INT_MAX).  tm: the maximum of the chunks that this
// thread read.  Chunk ch (eight logits) was read by thread ch % kT; run r of a thread is its
// `width` chunks from r * width on, with the (rounded up) maximum rmax[r][thread].
template <int DT>
__device__ void top_of(const typename Elem<DT>::type* z, int n, int top, float tm, const uint16_t (*rmax)[kT], int nruns,
                       int width, TopShared& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunks = (n + 7) >> 3, rounds = (chunks + kT - 1) / kT;
  const float pm = fmaxf(tm, __shfl_xor(tm, 1));
  __syncthreads();
  if ((tid & 1) == 0) sh.gm[tid >> 1] = pm;
  if (tid == 0) sh.nl = sh.ng = 0;
  __syncthreads();
  kth_pair(top, sh);
  __syncthreads();
  {
    const float tau = sh.tau;
    if (tm >= tau)
      for (int r = 0; r < nruns; ++r)
        if (__uint_as_float((uint32_t)rmax[r][tid] << 16) >= tau) {
          const int at = atomicAdd(&sh.nl, 1);
          if (at < kT) sh.runs[at] = (uint16_t)(r * kT + tid);
        }
    __syncthreads();
    const int nl = sh.nl;
    if (nl <= kT) {
      for (int f = tid; f < nl * width; f += kT) {
        const int e = f / width, run = sh.runs[e];
        const int j0 = (((run / kT) * width + f - e * width) * kT + run % kT) * 8;
        float v[8];
        if (j0 + 8 <= n) widen8<DT>(load_raw8<DT>(z + j0), v);
        else
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = j0 + j < n ? elem_to_f32<DT>(z[j0 + j]) : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (v[j] >= tau) {
            const int at = atomicAdd(&sh.ng, 1);
            if (at < kCand) {
              sh.cv[at] = v[j];
              sh.cj[at] = j0 + j;
            }
          }
      }
      __syncthreads();
      const int ng = sh.ng;
      if (ng <= kCand) {
        rank_top(ng, top, sh);
        // fewer only where the part has fewer logits
        for (int i = ng + tid; i < top; i += kT) {
          sh.cv[i] = -INFINITY;
          sh.cj[i] = 0x7FFFFFFF;
        }
        __syncthreads();
        return;
      }
    }
    __syncthreads();
  }
  for (;;) {
    const float tau = sh.tau;
    // the pairs to read again, in order (two waves' worth of flags)
    const bool in = tid < kPairs && sh.gm[tid < kPairs ? tid : 0] >= tau;
    const uint64_t mask = __ballot(in);
    if (lane == 0) sh.wsum[wave] = __popcll(mask);
    if (tid == 0) sh.ng = 0;
    __syncthreads();
    const int off = wave == 1 ? sh.wsum[0] : 0;
    if (in) sh.list[off + __popcll(mask & ((1ull << lane) - 1))] = (uint8_t)tid;
    const int nlist = 2 * (sh.wsum[0] + sh.wsum[1]);  // chunk columns: both threads of each pair
    int nt = 0;
    __syncthreads();
    // chunk `f` in order of ids: round f / nlist, the list's column f % nlist
    const int total = nlist * rounds;
    for (int f0 = 0; f0 < total; f0 += kT) {
      const int f = f0 + tid;
      float v[8];
      int j0 = n;
      if (f < total) {
        const int rd = f / nlist, col = f - rd * nlist;
        j0 = (rd * kT + sh.list[col >> 1] * 2 + (col & 1)) * 8;
      }
      int ties = 0;
      if (j0 + 8 <= n) widen8<DT>(load_raw8<DT>(z + j0), v);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j0 + j < n ? elem_to_f32<DT>(z[j0 + j]) : __uint_as_float(0x7FC00000u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (v[j] > tau) {
          const int at = atomicAdd(&sh.ng, 1);
          if (at < kCand) {
            sh.cv[at] = v[j];
            sh.cj[at] = j0 + j;
          }
        }
        ties += v[j] == tau ? 1 : 0;
      }
      // keep the first `top` equal ones: their places by a prefix sum over the workgroup
      if (nt < top && __syncthreads_or(ties)) {
        int run = ties;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int p = __shfl_up(run, o);
          if (lane >= o) run += p;
        }
        if (lane == 63) sh.wsum[wave] = run;
        __syncthreads();
        int at = nt + run - ties;
        int all = 0;
#pragma unroll
        for (int w = 0; w < kT / 64; ++w) {
          at += w < wave ? sh.wsum[w] : 0;
          all += sh.wsum[w];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (v[j] == tau) {
            if (at < top) sh.tie[at] = j0 + j;
            ++at;
          }
        nt = min(top, nt + all);
      }
    }
    __syncthreads();
    const int ng = sh.ng;
    if (ng <= kCand) {
      rank_top(ng, top, sh);
      for (int i = ng + tid; i < top; i += kT) {
        const bool have = i - ng < nt;
        sh.cv[i] = have ? tau : -INFINITY;
        sh.cj[i] = have ? sh.tie[i - ng] : 0x7FFFFFFF;
      }
      __syncthreads();
      return;
    }
    // Too many above the threshold (a few threads hold most large logits): the k-th largest of
    // those held is a higher threshold that still k logits reach; read again with that one.
    __syncthreads();
    kth_largest(sh.cv, kCand, top, sh);
    __syncthreads();
  }
}

// One part of one row (parts == 1: a whole row, finished here).
template <int DT>
__global__ __launch_bounds__(kT) void tok_kernel(TokArgs a, int parts, int seg, Part* __restrict__ ps,
                                                 float* __restrict__ pv, int* __restrict__ pj) {
  typedef typename Elem<DT>::type E;
  constexpr int kU = DT == W4_DT_F32 ? 2 : 4;  // chunks of eight a thread has in flight
  __shared__ Stat ws[kT / 64];
  __shared__ TopShared sh;
  __shared__ uint16_t rmax[kRuns][kT];
  const int64_t row = blockIdx.x / (unsigned)parts;
  const int part = blockIdx.x - (unsigned)row * parts;
  const int tid = threadIdx.x;
  const int j0 = part * seg;
  const int n = min(seg, (int)a.V - j0);
  const E* z = static_cast<const E*>(a.z) + row * a.ld + j0;
  const float c = a.inv_t * kLog2e;
  Stat st = {-INFINITY, 0.0f, 0.0f};
  Target target = {0, 0.0f};
  if (parts == 1 && tid == 0) target = load_target<DT>(a, row);
  // whole groups, the next one's loads in flight during the present one's exponentials
  const int groups = n / (kT * kU * 8);
  const int gpr = (groups + kRuns) / kRuns;  // groups a run (the rest counts as one)
  float run = -INFINITY;
  int left = gpr, r_at = 0;
  const E* p = z + tid * 8;
  Raw8<DT> next[kU];
  if (groups > 0)
#pragma unroll
    for (int u = 0; u < kU; ++u) next[u] = load_raw8<DT>(p + u * kT * 8);
  for (int g = 0; g < groups; ++g) {
    float v[kU * 8];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float w[8];
      widen8<DT>(next[u], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u * 8 + j] = w[j];
    }
    p += kT * kU * 8;
    if (g + 1 < groups)
#pragma unroll
      for (int u = 0; u < kU; ++u) next[u] = load_raw8<DT>(p + u * kT * 8);
    take(st, v, c, run);
    if (--left == 0) {
      rmax[r_at++][tid] = up16(run);
      run = -INFINITY;
      left = gpr;
    }
  }
  // the rest, chunk by chunk; logits past the end count as masked
  for (int j = groups * kT * kU * 8 + tid * 8; j < n; j += kT * 8) {
    float w[8];
    const uint32_t masked = DT == W4_DT_F32 ? 0xFF800000u : DT == W4_DT_F16 ? 0xFC00u : 0xFF80u;
    widen8<DT>(j + 8 <= n ? load_raw8<DT>(z + j) : load_raw8_part<DT>(z + j, n - j, masked), w);
    take(st, w, c, run);
  }
  rmax[r_at][tid] = up16(run);
  const float tm = st.m;
  st = wave_join(st, c);
  if ((tid & 63) == 0) ws[tid >> 6] = st;
  __syncthreads();
  st = ws[0];
#pragma unroll
  for (int w = 1; w < kT / 64; ++w) st = join(st, ws[w], c);
  const RowOut r = row_out(st);
  if (parts == 1) {
    if (tid == 0) write_row(a, row, r, target);
    if (a.top == 0) return;
    if (!r.bad) top_of<DT>(z, n, a.top, tm, rmax, r_at + 1, gpr * kU, sh);
    if (tid < a.top) {
      a.top_lp[row * a.top + tid] = r.bad ? r.mx : row_logprob(r, sh.cv[tid], a.inv_t);
      a.top_ids[row * a.top + tid] = r.bad ? -1 : sh.cj[tid];
    }
  } else {
    if (tid == 0) ps[blockIdx.x].st = st;
    if (a.top == 0 || r.bad) return;
    top_of<DT>(z, n, a.top, tm, rmax, r_at + 1, gpr * kU, sh);
    if (tid < a.top) {
      pv[(size_t)blockIdx.x * a.top + tid] = sh.cv[tid];
      pj[(size_t)blockIdx.x * a.top + tid] = sh.cj[tid] == 0x7FFFFFFF ? 0x7FFFFFFF : j0 + sh.cj[tid];
    }
  }
}

// Joins a row's parts: the statistics with one lane a part, then the alternatives from the
// parts' sorted lists.  The first ceil(top / parts) of each list are a pool of at least `top`
// logits, whose top-th largest is a threshold; what reaches it is ranked by counting.  Where
// that is too much (rows with very many equal logits), the lists are merged one by one: the
// parts are in order of ids, so of equal heads the lowest lane's goes first.  Entries that a
// short last part could not fill hold NaN, which no comparison or maximum takes.
template <int DT>
__global__ __launch_bounds__(kT) void tok_join_kernel(TokArgs a, int parts, const Part* __restrict__ ps,
                                                      const float* __restrict__ pv, const int* __restrict__ pj) {
  extern __shared__ float lists[];  // [parts][top] logits, then ids
  __shared__ TopShared sh;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const float c = a.inv_t * kLog2e;
  const int top = a.top, n = parts * top;
  const float nan = __uint_as_float(0x7FC00000u);
  int* ids = reinterpret_cast<int*>(lists + n);
  Stat st = {-INFINITY, 0.0f, 0.0f};
  Target target = {0, 0.0f};
  if (tid == 0) target = load_target<DT>(a, row);
  if (lane < parts) st = ps[(size_t)row * parts + lane].st;
#pragma unroll 4
  for (int i = tid; i < n; i += kT) {
    const int j = pj[(size_t)row * n + i];
    const float v = pv[(size_t)row * n + i];
    lists[i] = j == 0x7FFFFFFF ? nan : v;
    ids[i] = j;
  }
  const RowOut r = row_out(wave_join(st, c));
  if (tid == 0) write_row(a, row, r, target);
  if (top == 0) return;
  if (!r.bad) {
    __syncthreads();
    const int depth = (top + parts - 1) / parts, pool = parts * depth, pool4 = (pool + 3) & ~3;  // below 2 * 64
    if (tid < pool4) {
      const float v = tid < pool ? lists[tid / depth * top + tid % depth] : nan;
      sh.cv[tid] = v == v ? v : -INFINITY;
    }
    if (tid == 0) sh.ng = 0;
    __syncthreads();
    kth_largest(sh.cv, pool4, top, sh);
    __syncthreads();
    const float tau = sh.tau;
    for (int i = tid; i < n; i += kT)
      if (lists[i] >= tau) {
        const int at = atomicAdd(&sh.ng, 1);
        if (at < kCand) {
          sh.cv[at] = lists[i];
          sh.cj[at] = ids[i];
        }
      }
    __syncthreads();
    const int ng = sh.ng;
    if (ng <= kCand) {
      rank_top(ng, top, sh);
      __syncthreads();
    } else if (tid < 64) {
      int at = lane * top;
      const int end = lane < parts ? at + top : at;
      float v = at < end ? lists[at] : nan;
      for (int i = 0; i < top; ++i) {
        const float m = wave_max(__builtin_fmaxf(v, -INFINITY));  // NaN counts as -infinity here
        const int win = __ffsll((unsigned long long)__ballot(v == m)) - 1;
        if (lane == win) {
          sh.cv[i] = m;
          sh.cj[i] = ids[at];
          ++at;
          v = at < end ? lists[at] : nan;
        }
      }
    }
    if (tid >= 64) return;  // the first wave has written or (behind the barrier) sees the result
  }
  if (tid < top) {
    a.top_lp[row * top + tid] = r.bad ? r.mx : row_logprob(r, sh.cv[tid], a.inv_t);
    a.top_ids[row * top + tid] = r.bad ? -1 : sh.cj[tid];
  }
}

// Eight results as the logits' type, one store (two for fp32) at the element's alignment.
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::type* p, const float (&d)[8]) {
  typedef typename Elem<DT>::loose loose;
  u32x4 q[DT == W4_DT_F32 ? 2 : 1];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    if constexpr (DT == W4_DT_F32) {
      q[j >> 2][j & 3] = __float_as_uint(d[j]);
      q[j >> 2][(j & 3) + 1] = __float_as_uint(d[j + 1]);
    } else {
      q[0][j >> 1] = DT == W4_DT_F16 ? pack_f16x2(d[j], d[j + 1]) : pack_bf16x2(d[j], d[j + 1]);
    }
  }
  // written once and not read here again
  __builtin_nontemporal_store(q[0], reinterpret_cast<loose*>(p));
  if constexpr (DT == W4_DT_F32) __builtin_nontemporal_store(q[1], reinterpret_cast<loose*>(p + 4));
}

template <int DT>
__device__ __forceinline__ void store1(typename Elem<DT>::type* p, float d) {
  if constexpr (DT == W4_DT_F32) *p = d;
  else if constexpr (DT == W4_DT_F16) *p = f32_to_f16_bits(d);
  else *p = (uint16_t)(pack_bf16x2(d, 0.0f) & 0xFFFFu);
}

// Gradient of one part of a row: dz_j = -p_j (A + B log2 p_j) / T at every logit, with
// log2 p_j = (z_j - mx) c - L, then the few logits that have a gradient of their own (the
// target and the alternatives) written once more by the same workgroup.  Their logits are
// read before the part is written, so dz may be z.
template <int DT>
__global__ __launch_bounds__(kT) void tok_grad_kernel(TokGradArgs a, int parts, int seg) {
  typedef typename Elem<DT>::type E;
  constexpr int kU = DT == W4_DT_F32 ? 2 : 4;
  __shared__ float av[kMaxTop];
  __shared__ int aj[kMaxTop];
  const int64_t row = blockIdx.x / (unsigned)parts;
  const int part = blockIdx.x - (unsigned)row * parts;
  const int tid = threadIdx.x;
  const int j0 = part * seg;
  const int n = min(seg, (int)a.V - j0);
  const E* z = static_cast<const E*>(a.z) + row * a.ld + j0;
  E* dz = static_cast<E*>(a.dz) + row * a.ldd + j0;
  const float mx = a.stats[2 * row], logs = a.stats[2 * row + 1], ent = a.ent[row];
  const int64_t t = a.targets[row];
  const bool has_t = t != a.ignore && t >= 0 && t < a.V;
  const float g = has_t && a.g != nullptr ? a.g[row] : 0.0f;
  const float h = a.h != nullptr ? a.h[row] : 0.0f;
  const int top = a.a != nullptr ? a.top : 0;
  if (tid < top) {
    av[tid] = a.a[row * a.top + tid];
    aj[tid] = (int)a.top_ids[row * a.top + tid];
  }
  __syncthreads();
  float all = g;
  for (int i = 0; i < top; ++i) all += av[i];
  const bool empty = mx == -INFINITY;
  const float nan = mx != mx ? mx : 0.0f;  // a row that scored NaN has NaN gradients
  const float base = empty ? 0.0f : mx;
  const float c = a.inv_t * kLog2e, L = logs * kLog2e;
  // all + h (log p + ent), in units of log2 p, over T; an empty row has none
  const float A = empty ? 0.0f : (all + h * ent) * a.inv_t + nan, B = empty ? 0.0f : h * kLn2 * a.inv_t;
  auto at = [&](float v) {
    const float x = __builtin_fmaxf((v - base) * c - L, kFloor);
    return -__builtin_amdgcn_exp2f(x) * __builtin_fmaf(B, x, A);
  };
  // this thread's special logit, if it lies in this part: the target (thread 0) with what the
  // alternatives add to it, or an alternative that is not the target
  int sj = -1;
  float sg = 0.0f;
  if (tid == 0 && has_t) {
    sj = (int)t;
    sg = g;
    for (int i = 0; i < top; ++i) sg += aj[i] == sj ? av[i] : 0.0f;
  } else if (tid > 0 && tid <= top && !(has_t && aj[tid - 1] == t)) {
    sj = aj[tid - 1];
    sg = av[tid - 1];
  }
  sj -= j0;
  const bool special = sj >= 0 && sj < n && !empty;
  const float sz = special ? elem_to_f32<DT>(z[sj]) : 0.0f;
  __syncthreads();
  const int groups = n / (kT * kU * 8);
  const E* p = z + tid * 8;
  E* q = dz + tid * 8;
  Raw8<DT> next[kU];
  if (groups > 0)
#pragma unroll
    for (int u = 0; u < kU; ++u) next[u] = load_raw8<DT>(p + u * kT * 8);
  for (int i = 0; i < groups; ++i) {
    Raw8<DT> now[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) now[u] = next[u];
    p += kT * kU * 8;
    if (i + 1 < groups)
#pragma unroll
      for (int u = 0; u < kU; ++u) next[u] = load_raw8<DT>(p + u * kT * 8);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float w[8], d[8];
      widen8<DT>(now[u], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = at(w[j]);
      store8<DT>(q + u * kT * 8, d);
    }
    q += kT * kU * 8;
  }
  for (int j = groups * kT * kU * 8 + tid * 8; j < n; j += kT * 8) {
    if (j + 8 <= n) {
      float w[8], d[8];
      widen8<DT>(load_raw8<DT>(z + j), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = at(w[i]);
      store8<DT>(dz + j, d);
    } else {
      for (int i = j; i < n; ++i) store1<DT>(dz + i, at(elem_to_f32<DT>(z[i])));
    }
  }
  __syncthreads();
  if (special) store1<DT>(dz + sj, at(sz) + sg * a.inv_t);
}

// Parts of a row: one when the rows alone fill the device eight workgroups deep, else enough
// to come near that, of at least one chunk a thread (the launch that joins them takes one
// lane a part).
int parts_of(int64_t M, int64_t V, const DeviceCaps& caps, int most) {
  const int64_t want = (int64_t)caps.cus * 8;
  int64_t p = M >= want / 2 ? 1 : want / M;
  p = std::min<int64_t>(p, std::max<int64_t>(1, V / kMinSeg));
  return (int)std::min<int64_t>(p, most);
}
// Columns of a part: whole chunks, so that parts of aligned rows are aligned.
int seg_of(int64_t V, int parts) { return (int)(((V + parts - 1) / parts + 63) / 64 * 64); }

}  // namespace

size_t tok_ws_bytes(int64_t M, int64_t V, int top, const DeviceCaps& caps) {
  const int parts = parts_of(M, V, caps, kMaxParts);
  return parts == 1 ? 0 : (size_t)M * parts * (sizeof(Part) + 8 * (size_t)top);
}

// A launch holds fewer than 2^32 threads: rows are launched in runs of at most kRows.  How a row is
// cut is decided from all rows, as the workspace is, never from the rows of a run: a last run of
// few rows would take parts that no workspace was given for.
constexpr int64_t kRows = (int64_t)1 << 23;

static size_t elem_bytes(int dt) { return dt == W4_DT_F32 ? 4 : 2; }

hipError_t launch_tok(const TokArgs& all, const DeviceCaps& caps, void* ws, hipStream_t st) {
  TokArgs a = all;
  const int most = parts_of(all.M, all.V, caps, kMaxParts);
  const int seg = seg_of(all.V, most);
  const int parts = (int)((all.V + seg - 1) / seg);  // rounding the columns up may leave fewer
  // more than one part only of rows that are far fewer than kRows: one run
  Part* ps = most > 1 ? static_cast<Part*>(ws) : nullptr;
  float* pv = most > 1 ? reinterpret_cast<float*>(ps + (size_t)all.M * most) : nullptr;
  int* pj = most > 1 ? reinterpret_cast<int*>(pv + (size_t)all.M * parts * all.top) : nullptr;
  for (int64_t r = 0; r < all.M; r += kRows) {
    a.M = std::min(kRows, all.M - r);
    const unsigned g = (unsigned)(a.M * parts);
    switch (a.dt) {
      case W4_DT_F32: tok_kernel<W4_DT_F32><<<g, kT, 0, st>>>(a, parts, seg, ps, pv, pj); break;
      case W4_DT_F16: tok_kernel<W4_DT_F16><<<g, kT, 0, st>>>(a, parts, seg, ps, pv, pj); break;
      default: tok_kernel<W4_DT_BF16><<<g, kT, 0, st>>>(a, parts, seg, ps, pv, pj); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.z = static_cast<const char*>(a.z) + (size_t)(kRows * a.ld) * elem_bytes(a.dt);
    a.targets += kRows;
    a.lp += kRows;
    a.ent += kRows;
    a.stats += 2 * kRows;
    if (a.top > 0) {
      a.top_lp += kRows * a.top;
      a.top_ids += kRows * a.top;
    }
  }
  if (parts == 1) return hipSuccess;
  const size_t lds = (size_t)parts * all.top * 8;  // at most 64 x 64 pairs: 32 KB
  const unsigned g = (unsigned)all.M;
  switch (all.dt) {
    case W4_DT_F32: tok_join_kernel<W4_DT_F32><<<g, kT, lds, st>>>(all, parts, ps, pv, pj); break;
    case W4_DT_F16: tok_join_kernel<W4_DT_F16><<<g, kT, lds, st>>>(all, parts, ps, pv, pj); break;
    default: tok_join_kernel<W4_DT_BF16><<<g, kT, lds, st>>>(all, parts, ps, pv, pj); break;
  }
  return hipGetLastError();
}

hipError_t launch_tok_grad(const TokGradArgs& all, const DeviceCaps& caps, hipStream_t st) {
  TokGradArgs a = all;
  const int seg = seg_of(all.V, parts_of(all.M, all.V, caps, 1 << 20));
  const int parts = (int)((all.V + seg - 1) / seg);
  for (int64_t r = 0; r < all.M; r += kRows) {
    a.M = std::min(kRows, all.M - r);
    const unsigned g = (unsigned)(a.M * parts);
    switch (a.dt) {
      case W4_DT_F32: tok_grad_kernel<W4_DT_F32><<<g, kT, 0, st>>>(a, parts, seg); break;
      case W4_DT_F16: tok_grad_kernel<W4_DT_F16><<<g, kT, 0, st>>>(a, parts, seg); break;
      default: tok_grad_kernel<W4_DT_BF16><<<g, kT, 0, st>>>(a, parts, seg); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.z = static_cast<const char*>(a.z) + (size_t)(kRows * a.ld) * elem_bytes(a.dt);
    a.dz = static_cast<char*>(a.dz) + (size_t)(kRows * a.ldd) * elem_bytes(a.dt);
    a.targets += kRows;
    a.stats += 2 * kRows;
    a.ent += kRows;
    if (a.g != nullptr) a.g += kRows;
    if (a.h != nullptr) a.h += kRows;
    if (a.a != nullptr) {
      a.a += kRows * a.top;
      a.top_ids += kRows * a.top;
    }
  }
  return hipSuccess;
}

}  // namespace w4
