// C ABI of the microscaled 4-bit operators: argument validation, workspace layout, dispatch.  The
// contract of every entry point is in include/mxfp4.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/mxfp4.h"
#include "api_common.h"
#include "launch.h"

namespace {

using w4::aligned;
using w4::device_caps;
using w4::fail;
using w4::launched;
using w4::make_epi;
using w4::mx_pitch;
using w4::ok;

constexpr int64_t kMaxCols = (int64_t)1 << 22;       // 32-bit offsets in a tile of 256 rows
constexpr int64_t kMaxRows = ((int64_t)1 << 30) - 1;  // a launch holds fewer than 2^32 threads
constexpr int64_t kMaxGradN = (int64_t)1 << 20;      // the same of three parts of 16 bits
constexpr int64_t kMaxExpertWidth = (int64_t)1 << 17;
constexpr int64_t kDirectLd = (int64_t)1 << 22;

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
bool is_dtype(int d) { return d == W4_DT_F32 || d == W4_DT_F16 || d == W4_DT_BF16; }
size_t size_of(int d) { return d == W4_DT_F32 ? 4 : 2; }

int check_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0) return fail(W4_ERR_INVALID, "M = %lld must be >= 0", (long long)M);
  if (N < 1 || K < 1) return fail(W4_ERR_INVALID, "N = %lld and K = %lld must be >= 1", (long long)N, (long long)K);
  if (K >= kMaxCols) return fail(W4_ERR_UNSUPPORTED, "K = %lld must be below 2^22", (long long)K);
  if (M > kMaxRows || N > kMaxRows) return fail(W4_ERR_UNSUPPORTED, "M and N must be below 2^30");
  return W4_OK;
}

int check_mx(const uint8_t* codes, const uint8_t* scales) {
  if (!codes || !scales) return fail(W4_ERR_INVALID, "a required pointer is NULL");
  if (!aligned(codes, 16) || !aligned(scales, 4)) return fail(W4_ERR_ALIGN, "codes must be 16-byte, scales 4-byte aligned");
  return W4_OK;
}

int check_ws(const void* ws) {
  if (ws != nullptr && !aligned(ws, 16)) return fail(W4_ERR_ALIGN, "workspace must be 16-byte aligned");
  return W4_OK;
}

// Float rows: [rows][cols] of dtype, row stride ld.
int check_rows(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, const char* what) {
  if (!is_dtype(dtype)) return fail(W4_ERR_INVALID, "dtype = %d of %s is not F32, F16 or BF16", dtype, what);
  if (rows > 0 && X == nullptr) return fail(W4_ERR_INVALID, "%s is NULL", what);
  if (rows > 1 && ld < cols)
    return fail(W4_ERR_INVALID, "row stride %lld of %s is below its %lld columns", (long long)ld, what, (long long)cols);
  if (!aligned(X, size_of(dtype))) return fail(W4_ERR_ALIGN, "%s must be %zu-byte aligned", what, size_of(dtype));
  return W4_OK;
}

// Workspace of mx4_linear: the codes, the scales, then the product's own.
struct LinearWs {
  size_t scales, product, total;
};
LinearWs linear_ws(int64_t M, int64_t N, int64_t K) {
  LinearWs w;
  w.scales = up256((size_t)M * (mx_pitch(K) / 2));
  w.product = w.scales + up256((size_t)M * (mx_pitch(K) / 32));
  w.total = w.product + w4::mx_mm_workspace_bytes(M, N, K, device_caps());
  return w;
}

// Whether the input gradient reads bf16 parts of dY (or a copy, for bf16) at an aligned pitch, apart from
// a dY that is not 16-byte aligned.  ld < 0: the row stride is not known.
int64_t grad_pitch(int64_t N) { return (N + 63) / 64 * 64; }
bool grad_copies(int64_t M, int64_t N, int dtype, int64_t ld) {
  if (dtype != W4_DT_BF16 || ld < 0) return true;
  if (M <= 1) ld = N;
  return ld % 8 != 0 || N % 8 != 0 || ld >= kDirectLd;
}
size_t copy_bytes(int64_t M, int64_t N, int dtype) { return up256((size_t)M * w4::mx_parts(dtype) * grad_pitch(N) * 2); }

int check_moe(int64_t T, int64_t E, int top, int64_t H, int64_t F, int dtype) {
  if (!is_dtype(dtype)) return fail(W4_ERR_INVALID, "dtype = %d is not F32, F16 or BF16", dtype);
  if (T < 0 || E < 1 || H < 1 || F < 1)
    return fail(W4_ERR_INVALID, "T = %lld must be >= 0, E = %lld, H = %lld and F = %lld >= 1", (long long)T, (long long)E,
                (long long)H, (long long)F);
  if (top < 1 || top > E) return fail(W4_ERR_INVALID, "top = %d must be in [1, E = %lld]", top, (long long)E);
  if (E > w4::kMoeExperts || top > w4::kMoeTop)
    return fail(W4_ERR_UNSUPPORTED, "E = %lld and top = %d must be at most %d and %d", (long long)E, top, w4::kMoeExperts,
                w4::kMoeTop);
  if (H >= kMaxExpertWidth || F >= kMaxExpertWidth || T > kMaxRows)
    return fail(W4_ERR_UNSUPPORTED, "H and F must be below 2^17, T below 2^30");
  return W4_OK;
}

w4::MoeArgs moe_sizes(int64_t T, int64_t E, int top, int64_t H, int64_t F, int dtype) {
  w4::MoeArgs a = {};
  a.T = std::min<int64_t>(T, w4::kMoeTokens);
  a.E = E;
  a.top = top;
  a.H = H;
  a.F = F;
  a.dt = dtype;
  return a;
}
// A run's activations as bf16 parts, ahead of the layer's own workspace.
size_t moe_parts_bytes(const w4::MoeArgs& a) { return up256((size_t)a.T * w4::mx_parts(a.dt) * mx_pitch(a.H) * 2); }

}  // namespace

extern "C" {

int64_t mx4_pitch(int64_t cols) { return cols < 1 ? -1 : mx_pitch(cols); }

int mx4_quantize_rows(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales,
                      void* stream) {
  int s = check_sizes(rows, 1, cols);
  if (s != W4_OK) return s;
  s = check_rows(X, dtype, rows, cols, ld, "X");
  if (s != W4_OK) return s;
  if (rows == 0) return ok();
  s = check_mx(codes, scales);
  if (s != W4_OK) return s;
  if (rows == 1) ld = cols;
  return launched(w4::launch_mx_quantize(X, dtype, rows, cols, ld, codes, scales, static_cast<hipStream_t>(stream)),
                  "mx4_quantize_rows");
}

int mx4_dequantize_rows(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out, int out_dtype,
                        int64_t ldo, void* stream) {
  int s = check_sizes(rows, 1, cols);
  if (s != W4_OK) return s;
  s = check_rows(out, out_dtype, rows, cols, ldo, "out");
  if (s != W4_OK) return s;
  if (rows == 0) return ok();
  s = check_mx(codes, scales);
  if (s != W4_OK) return s;
  if (rows == 1) ldo = cols;
  return launched(w4::launch_mx_dequantize(codes, scales, rows, cols, out, out_dtype, ldo, static_cast<hipStream_t>(stream)),
                  "mx4_dequantize_rows");
}

int mx4_workspace_bytes(int64_t M, int64_t N, int64_t K, int x_dtype, size_t* bytes) {
  const int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  if (!bytes) return fail(W4_ERR_INVALID, "bytes is NULL");
  if (x_dtype >= 0 && !is_dtype(x_dtype)) return fail(W4_ERR_INVALID, "x_dtype = %d is unknown", x_dtype);
  if (M == 0) *bytes = 0;
  else if (x_dtype >= 0 && w4::mx_decode_supported(M, K)) *bytes = 0;
  else if (x_dtype < 0) *bytes = w4::mx_mm_workspace_bytes(M, N, K, device_caps());
  else *bytes = linear_ws(M, N, K).total;
  return ok();
}

int mx4_mm(const uint8_t* A, const uint8_t* a_scales, int64_t M, const uint8_t* W, const uint8_t* w_scales, int64_t N,
           int64_t K, const void* bias, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes,
           void* stream) {
  int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  w4::MxArgs a = {};
  s = make_epi(N, M, bias, out_dtype, segs, nsegs, &a.ep);
  if (s != W4_OK) return s;
  if (M == 0) return ok();
  s = check_mx(A, a_scales);
  if (s == W4_OK) s = check_mx(W, w_scales);
  if (s == W4_OK) s = check_ws(ws);
  if (s != W4_OK) return s;
  a.A = A;
  a.a_scales = a_scales;
  a.W = W;
  a.w_scales = w_scales;
  a.M = M;
  a.N = N;
  a.K = K;
  a.P = mx_pitch(K);
  return launched(w4::launch_mx_mm(a, device_caps(), ws, ws != nullptr ? ws_bytes : 0, static_cast<hipStream_t>(stream)),
                  "mx4_mm");
}

int mx4_linear(const void* X, int x_dtype, int64_t ldx, int64_t M, const uint8_t* W, const uint8_t* w_scales, int64_t N,
               int64_t K, const void* bias, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes,
               void* stream) {
  int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  s = check_rows(X, x_dtype, M, K, ldx, "X");
  if (s != W4_OK) return s;
  w4::Epi ep;
  s = make_epi(N, M, bias, out_dtype, segs, nsegs, &ep);
  if (s != W4_OK) return s;
  if (M == 0) return ok();
  s = check_mx(W, w_scales);
  if (s == W4_OK) s = check_ws(ws);
  if (s != W4_OK) return s;
  if (M == 1) ldx = K;
  if (w4::mx_decode_supported(M, K)) {
    w4::MxArgs a = {};
    a.X = X;
    a.x_dt = x_dtype;
    a.ldx = ldx;
    a.W = W;
    a.w_scales = w_scales;
    a.ep = ep;
    a.M = M;
    a.N = N;
    a.K = K;
    a.P = mx_pitch(K);
    return launched(w4::launch_mx_decode(a, device_caps(), static_cast<hipStream_t>(stream)), "mx4_linear");
  }
  const LinearWs l = linear_ws(M, N, K);
  if (ws == nullptr || ws_bytes < l.total)
    return fail(W4_ERR_RESOURCE, "mx4_linear needs a workspace of %zu bytes (got %zu)", l.total,
                ws != nullptr ? ws_bytes : (size_t)0);
  char* w = static_cast<char*>(ws);
  uint8_t* codes = reinterpret_cast<uint8_t*>(w);
  uint8_t* scales = reinterpret_cast<uint8_t*>(w + l.scales);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  s = launched(w4::launch_mx_quantize(X, x_dtype, M, K, ldx, codes, scales, st), "mx4_quantize_rows");
  if (s != W4_OK) return s;
  return mx4_mm(codes, scales, M, W, w_scales, N, K, bias, out_dtype, segs, nsegs, w + l.product, l.total - l.product,
                stream);
}

const char* mx4_kernel(int64_t M, int64_t N, int64_t K, int x_dtype) {
  if (check_sizes(M, N, K) != W4_OK || M == 0 || (x_dtype >= 0 && !is_dtype(x_dtype))) return nullptr;
  if (x_dtype >= 0 && w4::mx_decode_supported(M, K)) return "mx4_decode_fused";
  return w4::mx_mm_name(M, N, K, device_caps());
}

int mx4_mm_t_workspace_bytes(int64_t M, int64_t N, int64_t K, int dtype, int64_t ld, size_t* bytes) {
  const int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  if (!is_dtype(dtype)) return fail(W4_ERR_INVALID, "dtype = %d is not F32, F16 or BF16", dtype);
  if (N >= kMaxGradN) return fail(W4_ERR_UNSUPPORTED, "N = %lld must be below 2^20", (long long)N);
  if (!bytes) return fail(W4_ERR_INVALID, "bytes is NULL");
  *bytes = 0;
  if (M == 0) return ok();
  if (grad_copies(M, N, dtype, ld)) *bytes = copy_bytes(M, N, dtype);
  *bytes += w4::mx_grad_workspace_bytes(M, N, K, w4::mx_parts(dtype), device_caps());
  return ok();
}

int mx4_mm_t(const void* dY, int dtype, int64_t ld, int64_t M, const uint8_t* W, const uint8_t* w_scales, int64_t N,
             int64_t K, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes, void* stream) {
  int s = check_sizes(M, N, K);
  if (s != W4_OK) return s;
  s = check_rows(dY, dtype, M, N, ld, "dY");
  if (s != W4_OK) return s;
  w4::MxGradArgs a = {};
  s = make_epi(K, M, nullptr, out_dtype, segs, nsegs, &a.ep);
  if (s != W4_OK) return s;
  if (N >= kMaxGradN) return fail(W4_ERR_UNSUPPORTED, "N = %lld must be below 2^20", (long long)N);
  if (M == 0) return ok();
  s = check_mx(W, w_scales);
  if (s == W4_OK) s = check_ws(ws);
  if (s != W4_OK) return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (M == 1) ld = N;
  size_t wsb = ws != nullptr ? ws_bytes : 0;
  char* w = static_cast<char*>(ws);
  a.dY = static_cast<const uint16_t*>(dY);
  a.parts = w4::mx_parts(dtype);
  a.ld = ld;
  a.L = N;
  a.W = W;
  a.w_scales = w_scales;
  a.M = M;
  a.N = N;
  a.K = K;
  a.P = mx_pitch(K);
  if (grad_copies(M, N, dtype, ld) || !aligned(dY, 16)) {
    const size_t need = copy_bytes(M, N, dtype);
    if (wsb < need)
      return fail(W4_ERR_RESOURCE, "a dY of dtype %d, row stride %lld and %lld columns%s needs a workspace of %zu bytes (got %zu)",
                  dtype, (long long)ld, (long long)N, aligned(dY, 16) ? "" : ", not 16-byte aligned,", need, wsb);
    s = launched(w4::launch_mx_parts(dY, dtype, M, N, ld, grad_pitch(N), reinterpret_cast<uint16_t*>(w), st), "mx_parts");
    if (s != W4_OK) return s;
    a.dY = reinterpret_cast<const uint16_t*>(w);
    a.ld = a.L = grad_pitch(N);
    w += need;
    wsb -= need;
  }
  return launched(w4::launch_mx_grad(a, device_caps(), wsb > 0 ? w : nullptr, wsb, st), "mx4_mm_t");
}

int mx4_sum_workspace_bytes(int64_t M, int64_t N, size_t* bytes) {
  const int s = check_sizes(M, N, 1);
  if (s != W4_OK) return s;
  if (!bytes) return fail(W4_ERR_INVALID, "bytes is NULL");
  *bytes = w4::mx_sum_workspace_bytes(M, N, device_caps());
  return ok();
}

int mx4_sum_rows(const void* X, int dtype, int64_t M, int64_t N, int64_t ld, void* out, int out_dtype, void* ws, size_t ws_bytes,
                 void* stream) {
  int s = check_sizes(M, N, 1);
  if (s == W4_OK) s = check_rows(X, dtype, M, N, ld, "X");
  if (s == W4_OK) s = check_rows(out, out_dtype, 1, N, N, "out");
  if (s == W4_OK) s = check_ws(ws);
  if (s != W4_OK) return s;
  const w4_out_seg seg = {out, N, N};
  w4::Epi ep;
  s = make_epi(N, 1, nullptr, out_dtype, &seg, 1, &ep);
  if (s != W4_OK) return s;
  const w4::DeviceCaps caps = device_caps();
  const size_t need = w4::mx_sum_workspace_bytes(M, N, caps);
  if (need > 0 && (ws == nullptr || ws_bytes < need))
    return fail(W4_ERR_RESOURCE, "mx4_sum_rows needs a workspace of %zu bytes (got %zu)", need,
                ws != nullptr ? ws_bytes : (size_t)0);
  return launched(w4::launch_mx_sum(X, dtype, M, N, ld, ep, caps, ws, static_cast<hipStream_t>(stream)), "mx4_sum_rows");
}

int mx4_moe_workspace_bytes(int64_t T, int64_t E, int top, int64_t H, int64_t F, int dtype, size_t* bytes) {
  const int s = check_moe(T, E, top, H, F, dtype);
  if (s != W4_OK) return s;
  if (!bytes) return fail(W4_ERR_INVALID, "bytes is NULL");
  const w4::MoeArgs a = moe_sizes(T, E, top, H, F, dtype);
  *bytes = T == 0 ? 0 : moe_parts_bytes(a) + w4::moe_workspace_bytes(a, device_caps());
  return ok();
}

int mx4_moe(const void* X, int dtype, int64_t ldx, int64_t T, const void* logits, int logit_dtype, int64_t ldl, int64_t E,
            int top, int renorm, const uint8_t* W1, const uint8_t* w1_scales, const uint8_t* W2, const uint8_t* w2_scales,
            int64_t H, int64_t F, void* out, int64_t ldo, void* ws, size_t ws_bytes, void* stream) {
  int s = check_moe(T, E, top, H, F, dtype);
  if (s == W4_OK) s = check_rows(X, dtype, T, H, ldx, "X");
  if (s == W4_OK) s = check_rows(logits, logit_dtype, T, E, ldl, "logits");
  if (s == W4_OK) s = check_rows(out, dtype, T, H, ldo, "out");
  if (s != W4_OK) return s;
  if (T == 0) return ok();
  s = check_mx(W1, w1_scales);
  if (s == W4_OK) s = check_mx(W2, w2_scales);
  if (s == W4_OK) s = check_ws(ws);
  if (s != W4_OK) return s;
  if (T == 1) {
    ldx = H;
    ldl = E;
    ldo = H;
  }
  w4::MoeArgs a = moe_sizes(T, E, top, H, F, dtype);
  const w4::DeviceCaps caps = device_caps();
  const size_t parts = moe_parts_bytes(a), need = parts + w4::moe_workspace_bytes(a, caps);
  if (ws == nullptr || ws_bytes < need)
    return fail(W4_ERR_RESOURCE, "mx4_moe needs a workspace of %zu bytes (got %zu)", need, ws != nullptr ? ws_bytes : (size_t)0);
  a.renorm = renorm;
  a.ldt = logit_dtype;
  a.ldl = ldl;
  a.W1 = W1;
  a.w1_scales = w1_scales;
  a.W2 = W2;
  a.w2_scales = w2_scales;
  a.ldo = ldo;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  char* w = static_cast<char*>(ws);
  // bf16 rows of whole groups of 64 columns are read as they are, others through a copy at the pitch
  const bool direct = dtype == W4_DT_BF16 && H % 64 == 0 && ldx % 8 == 0 && ldx < kDirectLd && aligned(X, 16);
  for (int64_t t = 0; t < T; t += w4::kMoeTokens) {
    a.T = std::min<int64_t>(T - t, w4::kMoeTokens);
    const char* x = static_cast<const char*>(X) + (size_t)(t * ldx) * size_of(dtype);
    a.logits = static_cast<const char*>(logits) + (size_t)(t * ldl) * size_of(logit_dtype);
    a.out = static_cast<char*>(out) + (size_t)(t * ldo) * size_of(dtype);
    if (direct) {
      a.x = reinterpret_cast<const uint16_t*>(x);
      a.ldx = ldx;
      a.Hx = H;
    } else {
      s = launched(w4::launch_mx_parts(x, dtype, a.T, H, ldx, mx_pitch(H), reinterpret_cast<uint16_t*>(w), st), "mx_parts");
      if (s != W4_OK) return s;
      a.x = reinterpret_cast<const uint16_t*>(w);
      a.ldx = a.Hx = mx_pitch(H);
    }
    s = launched(w4::launch_moe(a, caps, w + parts, st), "mx4_moe");
    if (s != W4_OK) return s;
  }
  return ok();
}

}  // extern "C"
