/*
 * w8a8.h -- C ABI of the 8-bit integer linear operators and the token scores.
 *
 * Status codes, dtypes, output segments, ownership, streams and errors are those of
 * w4a16.h: every pointer is a device pointer owned by the caller (except the segment
 * array and the host out-parameters), arguments are validated on the host before any
 * launch, nothing is allocated or synchronized, and w4_last_error() holds the detail of
 * the last failure on the calling thread.
 *
 * Rows of int8 codes ("int8 rows"): R rows of C real columns, one fp32 scale per row.
 *   codes   int8 [R][P], P = w8_pitch(C) = C rounded up to a multiple of 64; the columns
 *           C .. P-1 of every row must be 0.  16-byte aligned.
 *   scales  fp32 [R]; the row stands for codes * scale.
 * Tokens and weight channels both use it: X [M][K] has one scale per token, W [N][K] one
 * per channel (output column).
 */
#ifndef W8A8_H
#define W8A8_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Row pitch, in bytes, of int8 rows with `cols` columns.  Host only; -1 if cols < 1. */
int64_t w8_pitch(int64_t cols);

/* Quantize X [rows][cols] (dtype F32, F16 or BF16, row stride ld >= cols elements, aligned
 * to the element) to int8 rows:
 *   a = max |x|,  s = max(fp32(a / 127), 2^-126),  q = rint(fp32(x * fp32(1 / s)))
 * in IEEE fp32, ties to even, so |q| <= 127 and |x - q s| <= s / 2 up to fp32 rounding.
 * The floor on s keeps 1 / s finite; a row of zeros gets codes 0.  A row that holds a NaN
 * or an infinity gets scale NaN and codes 0, so its products are NaN.  Columns
 * cols .. P-1 of codes are written as 0.  rows == 0 is a no-op; rows < 2^30, 1 <= cols < 2^17. */
int w8_quantize_rows(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, int8_t* codes, float* scales,
                     void* stream);

/* Device workspace, in bytes, of w8a8_mm (x_dtype < 0), w8a8_linear (x_dtype its activation
 * dtype) and w8a16_mm_t (for a dY of row stride ld, or any when ld < 0).  Host only. */
int w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K, int x_dtype, size_t* bytes);
int w8a16_mm_t_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t ld, size_t* bytes);

/* Y[m][n] = out_rne((fp32(sum_k A[m][k] W[n][k]) * w_scales[n]) * a_scales[m] + bias[n]) on
 * int8 rows A [M][K] and W [N][K]; the sum is exact in int32.  Output dtype, bias and
 * segments as for w4a16_mm_out (the segment columns sum to N).  M == 0 is a no-op.
 * M, N < 2^30, 1 <= K < 2^17.  The workspace is optional: with the bytes that w8a8_workspace_bytes
 * reports (16-byte aligned) a product with few output tiles splits its contraction; the
 * result is the same, bit for bit. */
int w8a8_mm(const int8_t* A, const float* a_scales, int64_t M, const int8_t* W, const float* w_scales, int64_t N,
            int64_t K, const void* bias, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes,
            void* stream);

/* w8a8_mm on float activations: X [M][K] (x_dtype F32, F16 or BF16, row stride ldx) is
 * quantized per token as by w8_quantize_rows and multiplied, with the same result as the
 * two calls.  Few tokens are quantized inside the product's launch.  The workspace that
 * w8a8_workspace_bytes reports is required (it holds the codes; 0 for few tokens). */
int w8a8_linear(const void* X, int x_dtype, int64_t ldx, int64_t M, const int8_t* W, const float* w_scales, int64_t N,
                int64_t K, const void* bias, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws,
                size_t ws_bytes, void* stream);

/* The input gradient of the product, on the same int8 rows W [N][K]:
 *   dX[m][k] = out_rne(sum_n dY[m][n] * w[n][k]),  w = rne16(W[n][k] * w_scales[n])
 * dY [M][N] BF16 or F16 (row stride ld), w rounded to dY's dtype (F16: to its eleven bits at any
 * size of the scales, down to channels whose scale is 2^-21 of the largest), fp32 accumulation.
 * The segments cover K columns.  N < 2^22, K < 2^17.  The workspace that
 * w8a16_mm_t_workspace_bytes reports is required when N or (for M > 1) ld is not a multiple
 * of 8, when ld is 2^22 or more, or when dY is not 16-byte aligned (it holds an aligned copy
 * of dY; for the last, ask with ld < 0), else optional (a split contraction, summed in a
 * fixed order). */
int w8a16_mm_t(const void* dY, int dtype, int64_t ld, int64_t M, const int8_t* W, const float* w_scales, int64_t N,
               int64_t K, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes, void* stream);

/* The same of an fp32 dY (row stride ld): w8a16_mm_t of F16 rows, each at a power of two that takes
 * its largest finite magnitude to [2^14, 2^15), the sums taken back by it exactly.  Eleven bits
 * of every dY down to 2^-29 of its row's largest; what is 2^-39 of it or less becomes 0.  The
 * workspace that w8a32_mm_t_workspace_bytes reports is required. */
int w8a32_mm_t_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes);
int w8a32_mm_t(const float* dY, int64_t ld, int64_t M, const int8_t* W, const float* w_scales, int64_t N, int64_t K,
               int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes, void* stream);

/* Name of the kernel w8a8_mm (x_dtype < 0) / w8a8_linear launches for these sizes, given
 * the workspace w8a8_workspace_bytes reports; NULL when they are invalid.  Host only. */
const char* w8a8_kernel(int64_t M, int64_t N, int64_t K, int x_dtype);

/* Scores of given tokens.  For row m of logits [M][V] (F32, F16 or BF16, row stride ld),
 * mx = max_j z_j, d_j = (z_j - mx) * fp32(1 / temperature), L = log sum_j exp(d_j), the log
 * probability of token j is d_j - L:
 *   logprobs[m]        that of targets[m];  0 where targets[m] == ignore, NaN where it is
 *                      outside [0, V) otherwise
 *   entropy[m]         -sum_j p_j log p_j, p = exp(d - L)  (nats)
 *   top_ids[m][i]      the `top` largest logits by (value, then the lower index),
 *   top_logprobs[m][i] and their log probabilities
 *   stats[m][0..1]     mx and L, kept for the gradient
 * A logit of -infinity has probability 0 (p log p = 0).  A row of only -infinity has no
 * distribution: logprobs and top_logprobs -infinity, entropy 0, stats -infinity and 0.  A
 * row with a NaN or +infinity: every float output NaN (logprobs 0 where ignored), top_ids -1.
 * 0 <= top <= min(V, 64); M, V <= 2^31 - 2^16; top outputs NULL when top == 0.  The workspace that
 * tok_workspace_bytes reports is required (0 when there are rows enough). */
int tok_workspace_bytes(int64_t M, int64_t V, int top, size_t* bytes);
int tok_logprobs(const void* logits, int dtype, int64_t M, int64_t V, int64_t ld, const int64_t* targets,
                 int64_t ignore, double temperature, int top, float* logprobs, float* entropy, float* stats,
                 float* top_logprobs, int64_t* top_ids, void* ws, size_t ws_bytes, void* stream);

/* Gradient of tok_logprobs with respect to the logits, for the gradients g (logprobs), h
 * (entropy) and a (top_logprobs; the ids held constant), any of which may be NULL (zero):
 *   dz_j = (g [j = target] + sum_i a_i [j = top_ids_i]
 *           - p_j (g + sum_i a_i + h (log p_j + entropy))) / temperature
 * rounded once to the logits' dtype.  g counts as 0 where the target is ignored or outside
 * [0, V).  A row of only -infinity gets 0, a row whose stats are NaN gets NaN.  dlogits
 * [M][V] (row stride ldd) may be the logits themselves (ldd == ld). */
int tok_logprobs_grad(const void* logits, int dtype, int64_t M, int64_t V, int64_t ld, const int64_t* targets,
                      int64_t ignore, double temperature, int top, const float* stats, const float* entropy,
                      const int64_t* top_ids, const float* g, const float* h, const float* a, void* dlogits,
                      int64_t ldd, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_H */
