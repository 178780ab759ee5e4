// Scores of given tokens (tok_logprobs) and their gradient, for gfx950.  For a row z of V
// logits, mx = max z, d = (z - mx) / T:
//   S = sum e^d,  logprob = d_t - log S,  entropy = log S - sum e^d d / S.
// The maximum is taken off before the division by T, so that nothing overflows (a mask of
// the type's lowest value divided by a small T) and the most likely tokens keep their bits.
#include "api_common.h"
#include "launch.h"
#include "rows.h"

namespace w4 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
// below this a term of the softmax is 0 in fp32: arguments are held above it, so that
// -infinity gives 0 and not infinity * 0
constexpr float kFloor = -1.0e4f;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <int T>
__device__ __forceinline__ float block_sum(float v, float* sh) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < T / 64; ++i) s += sh[i];
  return s;
}

constexpr int kT = 512;

// One workgroup a row; the alternatives one at a time, each the largest (value, lowest
// index) after the one before.
template <int DT>
__global__ __launch_bounds__(kT) void tok_kernel(TokArgs a) {
  typedef typename Elem<DT>::type E;
  __shared__ float sh[kT / 64];
  __shared__ int shi[kT / 64];
  const int64_t row = blockIdx.x;
  const E* z = static_cast<const E*>(a.z) + row * a.ld;
  const int V = (int)a.V;
  float mx = -INFINITY;
  int bad = 0;
  for (int j = threadIdx.x; j < V; j += kT) {
    const float v = elem_to_f32<DT>(z[j]);
    bad |= !(v < INFINITY);
    mx = fmaxf(mx, v);
  }
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kT / 64; ++i) mx = fmaxf(mx, sh[i]);
  const bool empty = mx == -INFINITY;
  if (empty) mx = 0.0f;
  float S = 0.0f, D = 0.0f;
  for (int j = threadIdx.x; j < V; j += kT) {
    const float d = fmaxf((elem_to_f32<DT>(z[j]) - mx) * a.inv_t, kFloor);
    const float e = __builtin_amdgcn_exp2f(d * kLog2e);
    S += e;
    D += e * d;
  }
  S = block_sum<kT>(S, sh);
  D = block_sum<kT>(D, sh);
  const float logs = logf(S);
  const float nan = __uint_as_float(0x7FC00000u);
  if (threadIdx.x == 0) {
    a.ent[row] = bad ? nan : empty ? 0.0f : logs - D / S;
    a.stats[2 * row] = bad ? nan : empty ? -INFINITY : mx;
    a.stats[2 * row + 1] = bad ? nan : empty ? 0.0f : logs;
    const int64_t t = a.targets[row];
    float lp;
    if (t == a.ignore) lp = 0.0f;
    else if (t < 0 || t >= V || bad) lp = nan;
    else lp = empty ? -INFINITY : (elem_to_f32<DT>(z[t]) - mx) * a.inv_t - logs;
    a.lp[row] = lp;
  }
  float last = INFINITY;
  int last_j = -1;
  for (int i = 0; i < a.top; ++i) {
    float bv = -INFINITY;
    int bj = 0x7FFFFFFF;
    for (int j = threadIdx.x; j < V; j += kT) {
      const float v = elem_to_f32<DT>(z[j]);
      const bool after = v < last || (v == last && j > last_j);
      if (after && (v > bv || (v == bv && j < bj))) {
        bv = v;
        bj = j;
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const float pv = __shfl_xor(bv, o);
      const int pj = __shfl_xor(bj, o);
      if (pv > bv || (pv == bv && pj < bj)) {
        bv = pv;
        bj = pj;
      }
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
      sh[threadIdx.x >> 6] = bv;
      shi[threadIdx.x >> 6] = bj;
    }
    __syncthreads();
    for (int w = 0; w < kT / 64; ++w)
      if (sh[w] > bv || (sh[w] == bv && shi[w] < bj)) {
        bv = sh[w];
        bj = shi[w];
      }
    last = bv;
    last_j = bj;
    if (threadIdx.x == 0) {
      a.top_ids[row * a.top + i] = bad ? -1 : bj;
      a.top_lp[row * a.top + i] = bad ? nan : empty ? -INFINITY : (bv - mx) * a.inv_t - logs;
    }
  }
}

template <int DT>
__device__ __forceinline__ typename Elem<DT>::type from_f32(float v) {
  if constexpr (DT == W4_DT_F32) return v;
  else if constexpr (DT == W4_DT_F16) return f32_to_f16_bits(v);
  else return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
}

template <int DT>
__global__ __launch_bounds__(kT) void tok_grad_kernel(TokGradArgs a) {
  typedef typename Elem<DT>::type E;
  const int64_t row = blockIdx.x;
  const E* z = static_cast<const E*>(a.z) + row * a.ld;
  E* dz = static_cast<E*>(a.dz) + row * a.ldd;
  const int V = (int)a.V;
  const float mx = a.stats[2 * row], logs = a.stats[2 * row + 1], ent = a.ent[row];
  const int64_t t = a.targets[row];
  const bool has_t = t != a.ignore && t >= 0 && t < V;
  const float g = has_t && a.g != nullptr ? a.g[row] : 0.0f;
  const float h = a.h != nullptr ? a.h[row] : 0.0f;
  float all = g;
  if (a.a != nullptr)
    for (int i = 0; i < a.top; ++i) all += a.a[row * a.top + i];
  for (int j = threadIdx.x; j < V; j += kT) {
    float d = 0.0f;
    if (mx != -INFINITY) {
      const float r = fmaxf((elem_to_f32<DT>(z[j]) - mx) * a.inv_t - logs, kFloor);
      d = -__builtin_amdgcn_exp2f(r * kLog2e) * (all + h * (r + ent));
      if (has_t && j == t) d += g;
      if (a.a != nullptr)
        for (int i = 0; i < a.top; ++i)
          if (a.top_ids[row * a.top + i] == j) d += a.a[row * a.top + i];
      d *= a.inv_t;
      if (mx != mx) d = mx;
    }
    dz[j] = from_f32<DT>(d);
  }
}

}  // namespace

size_t tok_ws_bytes(int64_t, int64_t, int, const DeviceCaps&) { return 0; }

hipError_t launch_tok(const TokArgs& a, const DeviceCaps&, void*, hipStream_t st) {
  const unsigned g = (unsigned)a.M;
  switch (a.dt) {
    case W4_DT_F32: tok_kernel<W4_DT_F32><<<g, kT, 0, st>>>(a); break;
    case W4_DT_F16: tok_kernel<W4_DT_F16><<<g, kT, 0, st>>>(a); break;
    default: tok_kernel<W4_DT_BF16><<<g, kT, 0, st>>>(a); break;
  }
  return hipGetLastError();
}

hipError_t launch_tok_grad(const TokGradArgs& a, const DeviceCaps&, hipStream_t st) {
  const unsigned g = (unsigned)a.M;
  switch (a.dt) {
    case W4_DT_F32: tok_grad_kernel<W4_DT_F32><<<g, kT, 0, st>>>(a); break;
    case W4_DT_F16: tok_grad_kernel<W4_DT_F16><<<g, kT, 0, st>>>(a); break;
    default: tok_grad_kernel<W4_DT_BF16><<<g, kT, 0, st>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace w4
