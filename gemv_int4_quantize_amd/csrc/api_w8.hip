// C ABI of the 8-bit integer linear operators and the token scores: argument validation,
// workspace layout, dispatch.  The contract of every entry point is in include/w8a8.h.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/w8a8.h"
#include "api_common.h"
#include "launch.h"

namespace {

using w4::aligned;
using w4::device_caps;
using w4::fail;
using w4::launched;
using w4::make_epi;
using w4::ok;

constexpr int64_t kMaxK = (int64_t)1 << 17;    // int32 sums: 128 * 128 * K < 2^31
constexpr int64_t kMaxScored = ((int64_t)1 << 31) - 65536;  // rows and columns of scores
constexpr int64_t kMaxRows = ((int64_t)1 << 30) - 1;   // a launch holds fewer than 2^32 threads
constexpr int64_t kMaxTop = 64;

int64_t pitch_of(int64_t cols) { return (cols + 63) / 64 * 64; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

bool is_dtype(int d) { return d == W4_DT_F32 || d == W4_DT_F16 || d == W4_DT_BF16; }
size_t size_of(int d) { return d == W4_DT_F32 ? 4 : 2; }

int check_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0) return fail(W4_ERR_INVALID, "M = %lld must be >= 0", (long long)M);
  if (N < 1 || K < 1) return fail(W4_ERR_INVALID, "N = %lld and K = %lld must be >= 1", (long long)N, (long long)K);
  if (K >= kMaxK) return fail(W4_ERR_UNSUPPORTED, "K = %lld must be below 2^17 (int32 sums)", (long long)K);
  if (M > kMaxRows || N > kMaxRows) return fail(W4_ERR_UNSUPPORTED, "M and N must be below 2^30");
  return W4_OK;
}

int check_weight(const int8_t* W, const float* w_scales) {
  if (!W || !w_scales) return fail(W4_ERR_INVALID, "a required pointer is NULL");
  if (!aligned(W, 16) || !aligned(w_scales, 4))
    return fail(W4_ERR_ALIGN, "codes must be 16-byte, scales 4-byte aligned");
  return W4_OK;
}

int check_ws(const void* ws) {
  if (ws != nullptr && !aligned(ws, 16)) return fail(W4_ERR_ALIGN, "workspace must be 16-byte aligned");
  return W4_OK;
}

// Float rows: [rows][cols] of dtype, row stride ld.
int check_rows(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, const char* what) {
  if (!is_dtype(dtype)) return fail(W4_ERR_INVALID, "dtype = %d is not F32, F16 or BF16", dtype);
  if (rows > 0 && X == nullptr) return fail(W4_ERR_INVALID, "%s is NULL", what);
  if (rows > 1 && ld < cols)
    return fail(W4_ERR_INVALID, "row stride %lld of %s is below its %lld columns", (long long)ld, what, (long long)cols);
  if (!aligned(X, size_of(dtype))) return fail(W4_ERR_ALIGN, "%s must be %zu-byte aligned", what, size_of(dtype));
  return W4_OK;
}

// Workspace of w8a8_linear: the codes, the scales, then the product's own.
struct LinearWs {
  size_t scales, product, total;
};
LinearWs linear_ws(int64_t M, int64_t N, int64_t K) {
  LinearWs w;
  w.scales = up256((size_t)M * pitch_of(K));
  w.product = w.scales + up256((size_t)M * 4);
  w.total = w.product + w4::w8_mm_workspace_bytes(M, N, K, device_caps());
  return w;
}

// Whether the input gradient reads a copy of dY's rows at an aligned pitch (apart from a dY that is
// not 16-byte aligned): 16-byte loads of every row, at 32-bit offsets in a tile of 256 rows.
// ld < 0: the row stride is not known.
constexpr int64_t kGradLd = (int64_t)1 << 22;
bool grad_copies(int64_t M, int64_t N, int64_t ld) {
  if (ld < 0) return true;
  if (M <= 1) ld = N;
  return ld % 8 != 0 || N % 8 != 0 || ld >= kGradLd;
}

// Workspace of w8a32_mm_t ahead of the product's own: fp16 rows, and their powers of two.
size_t half_bytes(int64_t M, int64_t N) { return up256((size_t)M * pitch_of(N) * 2) + up256((size_t)M * 4); }

}  // namespace

extern "C" {

int64_t w8_pitch(int64_t cols) { return cols < 1 ? -1 : pitch_of(cols); }

int w8_quantize_rows(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, int8_t* codes, float* scales,
                     void* stream) {
  int s = check_sizes(rows, 1, cols);
  if (s != W4_OK) return s;
  s = check_rows(X, dtype, rows, cols, ld, "X");
  if (s != W4_OK) return s;
  if (rows == 0) return ok();
  s = check_weight(codes, scales);
  if (s != W4_OK) return s;
  return launched(w4::launch_quantize_rows(X, dtype, rows, cols, ld, codes, scales, static_cast<hipStream_t>(stream)),
                  "quantize_rows");
}

int w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K, int x_dtype, size_t* bytes) {
  const int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  if (!bytes) return fail(W4_ERR_INVALID, "bytes is NULL");
  if (x_dtype >= 0 && !is_dtype(x_dtype)) return fail(W4_ERR_INVALID, "x_dtype = %d is unknown", x_dtype);
  if (M == 0) *bytes = 0;
  else if (x_dtype >= 0 && w4::w8_fused(M, K)) *bytes = 0;
  else if (x_dtype < 0) *bytes = w4::w8_mm_workspace_bytes(M, N, K, device_caps());
  else *bytes = linear_ws(M, N, K).total;
  return ok();
}

int w8a8_mm(const int8_t* A, const float* a_scales, int64_t M, const int8_t* W, const float* w_scales, int64_t N,
            int64_t K, const void* bias, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes,
            void* stream) {
  int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  w4::W8Args a = {};
  s = make_epi(N, M, bias, out_dtype, segs, nsegs, &a.ep);
  if (s != W4_OK) return s;
  if (M == 0) return ok();
  s = check_weight(A, a_scales);
  if (s == W4_OK) s = check_weight(W, w_scales);
  if (s == W4_OK) s = check_ws(ws);
  if (s != W4_OK) return s;
  a.A = A;
  a.a_scales = a_scales;
  a.W = W;
  a.w_scales = w_scales;
  a.M = M;
  a.N = N;
  a.K = K;
  a.pitch = pitch_of(K);
  return launched(w4::launch_w8_mm(a, device_caps(), ws, ws != nullptr ? ws_bytes : 0, static_cast<hipStream_t>(stream)),
                  "w8a8_mm");
}

int w8a8_linear(const void* X, int x_dtype, int64_t ldx, int64_t M, const int8_t* W, const float* w_scales, int64_t N,
                int64_t K, const void* bias, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws,
                size_t ws_bytes, void* stream) {
  int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  s = check_rows(X, x_dtype, M, K, ldx, "X");
  if (s != W4_OK) return s;
  w4::Epi ep;
  s = make_epi(N, M, bias, out_dtype, segs, nsegs, &ep);
  if (s != W4_OK) return s;
  if (M == 0) return ok();
  s = check_weight(W, w_scales);
  if (s == W4_OK) s = check_ws(ws);
  if (s != W4_OK) return s;
  if (w4::w8_fused(M, K)) {
    w4::W8Args a = {};
    a.X = X;
    a.x_dt = x_dtype;
    a.ldx = ldx;
    a.W = W;
    a.w_scales = w_scales;
    a.ep = ep;
    a.M = M;
    a.N = N;
    a.K = K;
    a.pitch = pitch_of(K);
    return launched(w4::launch_w8_decode(a, device_caps(), static_cast<hipStream_t>(stream)), "w8a8_linear");
  }
  const LinearWs l = linear_ws(M, N, K);
  if (ws == nullptr || ws_bytes < l.total)
    return fail(W4_ERR_RESOURCE, "w8a8_linear needs a workspace of %zu bytes (got %zu)", l.total,
                ws != nullptr ? ws_bytes : (size_t)0);
  char* w = static_cast<char*>(ws);
  int8_t* codes = reinterpret_cast<int8_t*>(w);
  float* scales = reinterpret_cast<float*>(w + l.scales);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  s = launched(w4::launch_quantize_rows(X, x_dtype, M, K, ldx, codes, scales, st), "quantize_rows");
  if (s != W4_OK) return s;
  return w8a8_mm(codes, scales, M, W, w_scales, N, K, bias, out_dtype, segs, nsegs, w + l.product,
                 l.total - l.product, stream);
}

const char* w8a8_kernel(int64_t M, int64_t N, int64_t K, int x_dtype) {
  if (check_sizes(M, N, K) != W4_OK || M == 0 || (x_dtype >= 0 && !is_dtype(x_dtype))) return nullptr;
  if (x_dtype >= 0 && w4::w8_fused(M, K)) return "w8_decode_fused";
  return w4::w8_mm_name(M, N, K, device_caps());
}

int w8a16_mm_t_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t ld, size_t* bytes) {
  const int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  if (!bytes) return fail(W4_ERR_INVALID, "bytes is NULL");
  *bytes = 0;
  if (M == 0) return ok();
  if (grad_copies(M, N, ld)) *bytes = up256((size_t)M * pitch_of(N) * 2);
  *bytes += w4::w8_grad_workspace_bytes(M, N, K, device_caps());
  return ok();
}

int w8a16_mm_t(const void* dY, int dtype, int64_t ld, int64_t M, const int8_t* W, const float* w_scales, int64_t N,
               int64_t K, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes, void* stream) {
  int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  if (dtype != W4_DT_F16 && dtype != W4_DT_BF16) return fail(W4_ERR_INVALID, "dtype = %d must be BF16 or F16", dtype);
  s = check_rows(dY, dtype, M, N, ld, "dY");
  if (s != W4_OK) return s;
  w4::Epi ep;
  s = make_epi(K, M, nullptr, out_dtype, segs, nsegs, &ep);
  if (s != W4_OK) return s;
  if (N >= kGradLd) return fail(W4_ERR_UNSUPPORTED, "N = %lld must be below 2^22", (long long)N);
  if (M == 0) return ok();
  s = check_weight(W, w_scales);
  if (s == W4_OK) s = check_ws(ws);
  if (s != W4_OK) return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (M == 1) ld = N;
  size_t wsb = ws != nullptr ? ws_bytes : 0;
  char* w = static_cast<char*>(ws);
  w4::W8GradArgs a = {static_cast<const uint16_t*>(dY), dtype == W4_DT_F16, ld, N, W, w_scales, ep, M, N, K, pitch_of(K), nullptr};
  if (grad_copies(M, N, ld) || !aligned(dY, 16)) {
    const int64_t npad = pitch_of(N);
    const size_t need = up256((size_t)M * npad * 2);
    if (wsb < need)
      return fail(W4_ERR_RESOURCE, "a dY of row stride %lld and %lld columns%s needs a workspace of %zu bytes (got %zu)",
                  (long long)ld, (long long)N, aligned(dY, 16) ? "" : ", not 16-byte aligned,", need, wsb);
    s = launched(w4::launch_pad_rows(static_cast<const uint16_t*>(dY), M, N, ld, reinterpret_cast<uint16_t*>(w), npad, st),
                 "pad_rows");
    if (s != W4_OK) return s;
    a.dY = reinterpret_cast<const uint16_t*>(w);
    a.ld = a.L = npad;
    w += need;
    wsb -= need;
  }
  return launched(w4::launch_w8_grad(a, device_caps(), wsb > 0 ? w : nullptr, wsb, st), "w8a16_mm_t");
}

int w8a32_mm_t_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  const int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  if (!bytes) return fail(W4_ERR_INVALID, "bytes is NULL");
  *bytes = M == 0 ? 0 : half_bytes(M, N) + w4::w8_grad_workspace_bytes(M, N, K, device_caps());
  return ok();
}

int w8a32_mm_t(const float* dY, int64_t ld, int64_t M, const int8_t* W, const float* w_scales, int64_t N, int64_t K,
               int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes, void* stream) {
  int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  s = check_rows(dY, W4_DT_F32, M, N, ld, "dY");
  if (s != W4_OK) return s;
  w4::Epi ep;
  s = make_epi(K, M, nullptr, out_dtype, segs, nsegs, &ep);
  if (s != W4_OK) return s;
  if (N >= kGradLd) return fail(W4_ERR_UNSUPPORTED, "N = %lld must be below 2^22", (long long)N);
  if (M == 0) return ok();
  s = check_weight(W, w_scales);
  if (s == W4_OK) s = check_ws(ws);
  if (s != W4_OK) return s;
  const size_t need = half_bytes(M, N);
  if (ws == nullptr || ws_bytes < need)
    return fail(W4_ERR_RESOURCE, "w8a32_mm_t needs a workspace of %zu bytes (got %zu)", need,
                ws != nullptr ? ws_bytes : (size_t)0);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t npad = pitch_of(N);
  char* w = static_cast<char*>(ws);
  uint16_t* half = reinterpret_cast<uint16_t*>(w);
  int* back = reinterpret_cast<int*>(w + up256((size_t)M * npad * 2));
  s = launched(w4::launch_half_rows(dY, M, N, ld, half, npad, back, st), "half_rows");
  if (s != W4_OK) return s;
  const w4::W8GradArgs a = {half, true, npad, npad, W, w_scales, ep, M, N, K, pitch_of(K), back};
  const size_t left = ws_bytes - need;
  return launched(w4::launch_w8_grad(a, device_caps(), left > 0 ? w + need : nullptr, left, st), "w8a32_mm_t");
}

int tok_workspace_bytes(int64_t M, int64_t V, int top, size_t* bytes) {
  if (M < 0 || V < 1 || top < 0 || top > kMaxTop || top > V)
    return fail(W4_ERR_INVALID, "M = %lld, V = %lld, top = %d: need M >= 0, V >= 1, 0 <= top <= min(V, %d)",
                (long long)M, (long long)V, top, (int)kMaxTop);
  if (V > kMaxScored || M > kMaxScored) return fail(W4_ERR_UNSUPPORTED, "M and V must fit in int32");
  if (!bytes) return fail(W4_ERR_INVALID, "bytes is NULL");
  *bytes = M == 0 ? 0 : w4::tok_ws_bytes(M, V, top, device_caps());
  return ok();
}

static int check_temperature(double t, float* inv) {
  *inv = (float)(1.0 / t);
  // the kernels scale by log2(e) / t as well
  if (!(t > 0.0) || !(*inv > 0.0f) || !std::isfinite(*inv * 1.5f))
    return fail(W4_ERR_INVALID, "temperature = %g must be positive with a finite fp32 reciprocal", t);
  return W4_OK;
}

int tok_logprobs(const void* logits, int dtype, int64_t M, int64_t V, int64_t ld, const int64_t* targets,
                 int64_t ignore, double temperature, int top, float* logprobs, float* entropy, float* stats,
                 float* top_logprobs, int64_t* top_ids, void* ws, size_t ws_bytes, void* stream) {
  size_t need = 0;
  int s = tok_workspace_bytes(M, V, top, &need);
  if (s != W4_OK) return s;
  s = check_rows(logits, dtype, M, V, ld, "logits");
  if (s != W4_OK) return s;
  w4::TokArgs a;
  s = check_temperature(temperature, &a.inv_t);
  if (s != W4_OK) return s;
  if (M == 0) return ok();
  if (!targets || !logprobs || !entropy || !stats || (top > 0 && (!top_logprobs || !top_ids)))
    return fail(W4_ERR_INVALID, "a required pointer is NULL");
  if (!aligned(targets, 8) || !aligned(top_ids, 8) || !aligned(logprobs, 4) || !aligned(entropy, 4) ||
      !aligned(stats, 4) || !aligned(top_logprobs, 4))
    return fail(W4_ERR_ALIGN, "targets and top_ids must be 8-byte, fp32 outputs 4-byte aligned");
  if (need > 0 && (ws == nullptr || ws_bytes < need))
    return fail(W4_ERR_RESOURCE, "tok_logprobs needs a workspace of %zu bytes (got %zu)", need,
                ws != nullptr ? ws_bytes : (size_t)0);
  s = check_ws(ws);
  if (s != W4_OK) return s;
  a.z = logits;
  a.dt = dtype;
  a.M = M;
  a.V = V;
  a.ld = ld;
  a.targets = targets;
  a.ignore = ignore;
  a.top = top;
  a.lp = logprobs;
  a.ent = entropy;
  a.stats = stats;
  a.top_lp = top_logprobs;
  a.top_ids = top_ids;
  return launched(w4::launch_tok(a, device_caps(), ws, static_cast<hipStream_t>(stream)), "tok_logprobs");
}

int tok_logprobs_grad(const void* logits, int dtype, int64_t M, int64_t V, int64_t ld, const int64_t* targets,
                      int64_t ignore, double temperature, int top, const float* stats, const float* entropy,
                      const int64_t* top_ids, const float* g, const float* h, const float* a_top, void* dlogits,
                      int64_t ldd, void* stream) {
  size_t need = 0;
  int s = tok_workspace_bytes(M, V, top, &need);
  if (s != W4_OK) return s;
  s = check_rows(logits, dtype, M, V, ld, "logits");
  if (s == W4_OK) s = check_rows(dlogits, dtype, M, V, ldd, "dlogits");
  if (s != W4_OK) return s;
  w4::TokGradArgs a;
  s = check_temperature(temperature, &a.inv_t);
  if (s != W4_OK) return s;
  if (M == 0) return ok();
  if (!targets || !stats || !entropy || (top > 0 && a_top != nullptr && !top_ids))
    return fail(W4_ERR_INVALID, "a required pointer is NULL");
  if (!aligned(targets, 8) || !aligned(top_ids, 8) || !aligned(stats, 4) || !aligned(entropy, 4) || !aligned(g, 4) ||
      !aligned(h, 4) || !aligned(a_top, 4))
    return fail(W4_ERR_ALIGN, "targets and top_ids must be 8-byte, fp32 inputs 4-byte aligned");
  if (logits == dlogits && M > 1 && ld != ldd)
    return fail(W4_ERR_INVALID, "in place, ldd = %lld must be ld = %lld", (long long)ldd, (long long)ld);
  a.z = logits;
  a.dt = dtype;
  a.M = M;
  a.V = V;
  a.ld = ld;
  a.targets = targets;
  a.ignore = ignore;
  a.top = top;
  a.stats = stats;
  a.ent = entropy;
  a.top_ids = top_ids;
  a.g = g;
  a.h = h;
  a.a = top > 0 ? a_top : nullptr;
  a.dz = dlogits;
  a.ldd = ldd;
  return launched(w4::launch_tok_grad(a, device_caps(), static_cast<hipStream_t>(stream)), "tok_logprobs_grad");
}

}  // extern "C"
