/*
 * mxfp4.h -- C ABI of the microscaled 4-bit (MXFP4) operators.
 *
 * Status codes, dtypes, output segments, ownership, streams and errors are those of
 * w4a16.h: every pointer is a device pointer owned by the caller (except the segment
 * array and the host out-parameters), arguments are validated on the host before any
 * launch, nothing is allocated or synchronized, and w4_last_error() holds the detail of
 * the last failure on the calling thread.
 *
 * Rows of microscaled codes ("mx4 rows", the MXFP4 format of the OCP microscaling
 * specification): R rows of C real columns, padded to P = mx4_pitch(C), C rounded up to a
 * multiple of 128.
 *   codes   uint8 [R][P / 2], 16-byte aligned: column 2j in the low four bits of byte j, column
 *           2j + 1 in the high ones.  A code is e2m1: sign, two exponent bits, one mantissa
 *           bit, for 0, .5, 1, 1.5, 2, 3, 4, 6.  The codes of columns C .. P-1 must be 0.
 *   scales  uint8 [R][P / 32], 4-byte aligned: every 32 columns share 2^(scale - 127); 255: NaN.
 *           Blocks of nothing but columns C .. P-1 may have any scale but 255, which would make the
 *           products of their row NaN (the quantizer writes 0).
 * Tokens and weight channels both use it: X [M][K] is quantized along K, W [N][K] as well.
 * Rows, M and N are below 2^30, columns and K below 2^22.  Outputs overlap no input.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns that a row of `cols` is padded to.  Host only; -1 if cols < 1. */
int64_t mx4_pitch(int64_t cols);

/* Quantize X [rows][cols] (dtype F32, F16 or BF16, row stride ld >= cols elements, aligned to the
 * element) to mx4 rows: for each block of 32 columns, a = max |x|,
 *   scale = max(floor(log2 a) - 2 + 127, 0),  code = x / 2^(scale - 127) rounded to e2m1,
 * ties to the even code, magnitudes above 6 to 6; the sign is x's.  A block of zeros has scale 0.  A
 * block with a NaN or an infinity has scale 255 and codes 0, so that what it enters is NaN.
 * Padding gets codes 0.  rows == 0 is a no-op. */
int mx4_quantize_rows(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales,
                      void* stream);

/* out [rows][cols] (out_dtype F32, F16 or BF16, row stride ldo) = code * 2^(scale - 127): exact in
 * F32 and BF16 (magnitudes past the type's largest are infinite), rounded to nearest even in F16. */
int mx4_dequantize_rows(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out, int out_dtype,
                        int64_t ldo, void* stream);

/* Device workspace, in bytes, of mx4_mm (x_dtype < 0) and mx4_linear (x_dtype its activation dtype).
 * Host only. */
int mx4_workspace_bytes(int64_t M, int64_t N, int64_t K, int x_dtype, size_t* bytes);

/* Y[m][n] = out_rne(sum_k a[m][k] w[n][k] + bias[n]) on mx4 rows A [M][K] and W [N][K]: exact products,
 * fp32 sums, the bias added in fp32, one rounding.  Output dtype, bias and segments as for
 * w4a16_mm_out (the segment columns sum to N).  M == 0 is a no-op.  The workspace is optional: with
 * the bytes that mx4_workspace_bytes reports (16-byte aligned) a product with few output tiles
 * splits its contraction, in a fixed order of sums. */
int mx4_mm(const uint8_t* A, const uint8_t* a_scales, int64_t M, const uint8_t* W, const uint8_t* w_scales, int64_t N,
           int64_t K, const void* bias, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes,
           void* stream);

/* mx4_mm on float activations: X [M][K] (x_dtype F32, F16 or BF16, row stride ldx) is quantized as by
 * mx4_quantize_rows and multiplied.  Few tokens are quantized inside the product's launch.  The
 * workspace that mx4_workspace_bytes reports is required (it holds the codes; 0 for few tokens). */
int mx4_linear(const void* X, int x_dtype, int64_t ldx, int64_t M, const uint8_t* W, const uint8_t* w_scales, int64_t N,
               int64_t K, const void* bias, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes,
               void* stream);

/* Name of the kernel mx4_mm (x_dtype < 0) / mx4_linear launches for these sizes, given the workspace
 * mx4_workspace_bytes reports; NULL when they are invalid.  Host only. */
const char* mx4_kernel(int64_t M, int64_t N, int64_t K, int x_dtype);

/* The input gradient of the product, on the same mx4 rows W [N][K]:
 *   dX[m][k] = out_rne(sum_n dY[m][n] w[n][k])
 * dY [M][N] BF16, F16 or F32 (row stride ld), w and dY as they are (w in bf16's range, 2^128), fp32
 * sums, one rounding.  The segments cover K columns.  N < 2^20.  The workspace that
 * mx4_mm_t_workspace_bytes reports (ld < 0: for any dY) is required for F16 and F32 (bf16 parts of
 * dY: two and three), and for a BF16 dY whose N or (for M > 1) ld is not a multiple of 8, whose ld is
 * 2^22 or more or that is not 16-byte aligned (a copy; for the last, ask with ld < 0); else it is
 * optional (a split contraction, summed in a fixed order). */
int mx4_mm_t_workspace_bytes(int64_t M, int64_t N, int64_t K, int dtype, int64_t ld, size_t* bytes);
int mx4_mm_t(const void* dY, int dtype, int64_t ld, int64_t M, const uint8_t* W, const uint8_t* w_scales, int64_t N,
             int64_t K, int out_dtype, const w4_out_seg* segs, int nsegs, void* ws, size_t ws_bytes, void* stream);

/* out[n] = out_rne(sum_m X[m][n]): X [M][N] F32, F16 or BF16 (row stride ld), out [N] of out_dtype; the bias's
 * gradient of a linear layer, from dY.  fp32 sums in an order that M and N fix.  M == 0: zeros.  The
 * workspace that mx4_sum_workspace_bytes reports is required. */
int mx4_sum_workspace_bytes(int64_t M, int64_t N, size_t* bytes);
int mx4_sum_rows(const void* X, int dtype, int64_t M, int64_t N, int64_t ld, void* out, int out_dtype, void* ws, size_t ws_bytes,
                 void* stream);

/* A mixture-of-experts layer for few tokens.  For token t (x = X[t], z = logits[t]) and the `top` experts
 * with the largest logits, by value and then the lower index:
 *   a_j = silu(G_j x) * (U_j x),  out[t] = sum_j g_j D_j a_j,  g_j = exp(z_j - max z) / total
 * total the sum of exp(z_i - max z) over the chosen experts (renorm != 0) or over all E.  Expert e's gate
 * G_e is rows 2 F e .. 2 F e + F - 1 of the mx4 rows W1 [E * 2F][H], its up projection U_e the next F,
 * and D_e is rows e H .. e H + H - 1 of W2 [E * H][F].  X [T][H] has dtype F32, F16 or BF16 and row
 * stride ldx, out the same dtype and row stride ldo; logits [T][E] any of the three, row stride ldl.
 * The weights and x enter as they are, sums, a_j and g_j are fp32, and so is g_j a_j between the two
 * products; one rounding of the result.
 * A logit of -infinity is an expert that is masked: it is never run, also where fewer than `top` are
 * left.  A token whose logits are all -infinity gets 0.  A token with a NaN or +infinity among its
 * logits gets NaN.
 * 1 <= top <= min(E, 16), E <= 512, H and F < 2^17.  T == 0 is a no-op; more than 64 tokens run 64 at a time,
 * each run reading its weights again.  The workspace that mx4_moe_workspace_bytes reports is
 * required; it belongs to the call until its launches have ended. */
int mx4_moe_workspace_bytes(int64_t T, int64_t E, int top, int64_t H, int64_t F, int dtype, size_t* bytes);
int mx4_moe(const void* X, int dtype, int64_t ldx, int64_t T, const void* logits, int logit_dtype, int64_t ldl, int64_t E,
            int top, int renorm, const uint8_t* W1, const uint8_t* w1_scales, const uint8_t* W2, const uint8_t* w2_scales,
            int64_t H, int64_t F, void* out, int64_t ldo, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
