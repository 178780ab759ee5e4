// Internal launchers of the W4A16 library (host side).  Arguments are validated
// by the C ABI layer before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/w4a16.h"

namespace w4 {

// intz: integer zero points (z = clamp(rint(-min / s), 0, 15), q = clamp(rint(w / s) + z, 0, 15))
hipError_t launch_quantize(const void* W, int dt, int64_t N, int64_t K, int mode, int g, int intz, int32_t* packed,
                           uint16_t* scales, uint16_t* zeros, void* ws, hipStream_t st);
size_t quantize_workspace_bytes(int mode);

hipError_t launch_dequantize(const int32_t* packed, const uint16_t* scales, const uint16_t* zeros, int64_t N,
                             int64_t K, int mode, int g, void* out, int out_dt, hipStream_t st);

// Output epilogue of a matmul (passed to the kernels by value): output column c of
// row m gets out_rne(acc + bias[c]) in dtype dt, stored in the segment s holding c at
// y[s] + m * ld[s] + (c - c0[s]).  The bias, when present, has the output dtype.
constexpr int kMaxSegs = 4;
struct Epi {
  const void* bias;             // nullptr or [outc] elements of dt
  int dt;                       // W4_DT_F32, W4_DT_F16 or W4_DT_BF16
  int nseg;                     // 1 .. kMaxSegs
  int64_t c0[kMaxSegs];         // first column of each segment (INT64_MAX past nseg)
  void* y[kMaxSegs];
  int64_t ld[kMaxSegs];         // row stride of each segment, in elements
};

// Matmul problem after validation: A [M][L] bf16 (L = contraction), packed [N][K/8].
struct MmArgs {
  const uint16_t* A;
  const int32_t* packed;
  const uint16_t* scales;
  const uint16_t* zeros;
  Epi ep;
  int64_t M, N, K;
  int mode;   // w4_mode
  int group;  // GROUPWISE g, else K
  bool transposed;
  bool a_f16;  // activations (and the weight operand) fp16 instead of bf16
};

// Properties of the current device that kernel plans depend on.
struct DeviceCaps {
  size_t lds;  // dynamic LDS bytes one workgroup may use
  int cus;     // compute units
};

// GEMV (M <= 4, non-transposed).  Returns false if this shape cannot run on it
// (LDS footprint), so the caller can fall back to the GEMM.
bool gemv_supported(const MmArgs& a, const DeviceCaps& caps);
const char* gemv_name(const MmArgs& a);
size_t gemv_lds_bytes(const MmArgs& a, const DeviceCaps& caps);
hipError_t launch_gemv(const MmArgs& a, const DeviceCaps& caps, hipStream_t st);

// GEMM: the workspace the split-K plan wants (0 if none), and for a launch given a
// workspace of ws_bytes (0: none) the plan it runs -- split only when ws_bytes holds the
// split plan's bytes: its kernel name (with a split-K or split-tail suffix), the LDS bytes
// of its tile and the workspace bytes it uses.  launch_gemm runs that same plan.
size_t gemm_workspace_bytes(const MmArgs& a, const DeviceCaps& caps);
const char* gemm_name(const MmArgs& a, const DeviceCaps& caps, size_t ws_bytes);
size_t gemm_lds_bytes(const MmArgs& a, const DeviceCaps& caps, size_t ws_bytes);
size_t gemm_used_workspace_bytes(const MmArgs& a, const DeviceCaps& caps, size_t ws_bytes);
hipError_t launch_gemm(const MmArgs& a, const DeviceCaps& caps, void* ws, size_t ws_bytes, hipStream_t st);

// The part of a GEMM one launch covers: output column tiles [ct0, ct0 + nct) (nct = 0:
// all of them from ct0 on), with the contraction cut into `splits` slices.  With
// splits > 1 each slice writes its fp32 partial sums to its own plane of the workspace,
// [M][pw] where pw is the number of covered columns (column ct0 * BN first), and a
// reduction finishes them through the output epilogue.
struct GemmPart {
  int splits = 1;
  int ct0 = 0, nct = 0;
};

// Non-transposed GEMM with the weight operand dequantized into MFMA registers
// (tile 0: 128 x 128, 1: 256 x 128, 2: 64 x 128, 3: 32 x 128).
bool gemm_nt_reg_supported(const MmArgs& a);
hipError_t launch_gemm_nt_reg(const MmArgs& a, int tile, const GemmPart& gp, float* part, hipStream_t st);

// Mid-M forward matmul (kSkinnyMinM <= M <= kSkinnyMaxM) on 16x16x32 MFMAs with the
// activations held in registers (skinny.hip).  A plan covers the rows in `blocks` blocks of
// `rpb` rows and the contraction in `splits` ranges of `units_per_split` 128-column units;
// with splits > 1 the sums go to [splits][M][N] fp32 planes and the split-K reduction
// finishes them.  ok = false: this problem does not fit the kernel (the GEMM tiles run).
constexpr int kSkinnyMinM = 5, kSkinnyMaxM = 32;
struct SkinnyPlan {
  bool ok = false;
  int MB = 1, UP = 1;  // 16-row blocks of X; 128-column units per wave
  int splits = 1, units_per_split = 0;
  int rpb = 0, blocks = 0;
  int log2gr = 0;  // the partial sums are reduced in rounds of 2^log2gr 16-row groups
  size_t lds = 0;
};
bool skinny_supported(const MmArgs& a);
SkinnyPlan skinny_plan(const MmArgs& a, const DeviceCaps& caps, bool allow_split);
size_t skinny_split_bytes(const MmArgs& a, const SkinnyPlan& p);
const char* skinny_name(const MmArgs& a, const SkinnyPlan& p);
hipError_t launch_skinny(const MmArgs& a, const SkinnyPlan& p, float* part, hipStream_t st);

// Output columns [c_lo, c_lo + pw) = epilogue(sum of `splits` fp32 [M][pw] planes, in a
// fixed order).
hipError_t launch_splitk_reduce(const float* part, int splits, int64_t M, int64_t c_lo, int64_t pw, const Epi& ep,
                                hipStream_t st);

// ---- 8-bit integer linear operators (include/w8a8.h)

// X [rows][cols] (dtype dt, row stride ld) -> codes [rows][pitch], scales [rows].
hipError_t launch_quantize_rows(const void* X, int dt, int64_t rows, int64_t cols, int64_t ld, int8_t* codes,
                                float* scales, hipStream_t st);

// Product of int8 rows after validation.  X != nullptr: float activations (dtype x_dt, row
// stride ldx) that the decode kernel quantizes itself; else A / a_scales.
struct W8Args {
  const int8_t* A;
  const float* a_scales;
  const void* X;
  int x_dt;
  int64_t ldx;
  const int8_t* W;
  const float* w_scales;
  Epi ep;
  int64_t M, N, K, pitch;
};
size_t w8_mm_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps);
const char* w8_mm_name(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps);
hipError_t launch_w8_mm(const W8Args& a, const DeviceCaps& caps, void* ws, size_t ws_bytes, hipStream_t st);
// Few tokens (w8_decode.hip); w8_fused: float tokens are quantized inside that launch.
bool w8_fused(int64_t M, int64_t K);
bool w8_decode_supported(int64_t M);
hipError_t launch_w8_decode(const W8Args& a, const DeviceCaps& caps, hipStream_t st);

// Input gradient (w8_grad.hip): dY [M][N] 16-bit, row stride ld (a multiple of 8, as N), 16-byte
// aligned.  L: columns of dY to read, N or (zeros past N) N rounded up to 64.
struct W8GradArgs {
  const uint16_t* dY;
  bool f16;
  int64_t ld, L;
  const int8_t* W;
  const float* w_scales;
  Epi ep;
  int64_t M, N, K, pitch;
  const int* back;  // F16: powers of two that the rows' sums are multiplied by (or nullptr)
};
size_t w8_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps);
hipError_t launch_w8_grad(const W8GradArgs& a, const DeviceCaps& caps, void* ws, size_t ws_bytes, hipStream_t st);

// X [rows][cols] fp32, row stride ld -> out [rows][pitch] fp16 of X times 2^-back[row] (w8_quantize.hip).
hipError_t launch_half_rows(const float* X, int64_t rows, int64_t cols, int64_t ld, uint16_t* out, int64_t pitch,
                            int* back, hipStream_t st);

// dY [M][N] 16-bit, row stride ld -> out [M][npad], zeros past column N.
hipError_t launch_pad_rows(const uint16_t* dY, int64_t M, int64_t N, int64_t ld, uint16_t* out, int64_t npad,
                           hipStream_t st);

// ---- microscaled 4-bit operators (include/mxfp4.h)

constexpr int64_t mx_pitch(int64_t cols) { return (cols + 127) / 128 * 128; }

// X [rows][cols] (dtype dt, row stride ld) -> codes [rows][P / 2], scales [rows][P / 32], and back.
hipError_t launch_mx_quantize(const void* X, int dt, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                              uint8_t* scales, hipStream_t st);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out, int dt,
                                int64_t ldo, hipStream_t st);

// X [rows][cols] -> out [rows][mx_parts(dt)][pitch] bf16, parts whose sum is X, zeros past the columns.
constexpr int mx_parts(int dt) { return dt == W4_DT_F32 ? 3 : dt == W4_DT_F16 ? 2 : 1; }
hipError_t launch_mx_parts(const void* X, int dt, int64_t rows, int64_t cols, int64_t ld, int64_t pitch, uint16_t* out,
                           hipStream_t st);

// Product of microscaled rows after validation.  X != nullptr: float activations (dtype x_dt, row
// stride ldx) that the decode kernel quantizes itself; else A / a_scales.  P: padded columns.
struct MxArgs {
  const uint8_t* A;
  const uint8_t* a_scales;
  const void* X;
  int x_dt;
  int64_t ldx;
  const uint8_t* W;
  const uint8_t* w_scales;
  Epi ep;
  int64_t M, N, K, P;
};
size_t mx_mm_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps);
const char* mx_mm_name(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps);
hipError_t launch_mx_mm(const MxArgs& a, const DeviceCaps& caps, void* ws, size_t ws_bytes, hipStream_t st);
// Few tokens (mx_decode.hip): float ones, quantized inside that launch, or one or two of ready codes.
bool mx_decode_supported(int64_t M, int64_t K);
bool mx_decode_ready_supported(int64_t M, int64_t K);
hipError_t launch_mx_decode(const MxArgs& a, const DeviceCaps& caps, hipStream_t st);
// More of ready codes.
bool mx_few_supported(int64_t M, int64_t N, int64_t K, const DeviceCaps& caps);
hipError_t launch_mx_few(const MxArgs& a, const DeviceCaps& caps, hipStream_t st);

// Input gradient (mx_grad.hip): dY [M][parts][ld] bf16 parts (ld a multiple of 8, L <= ld columns of
// each to read), 16-byte aligned.
struct MxGradArgs {
  const uint16_t* dY;
  int parts;
  int64_t ld, L;
  const uint8_t* W;
  const uint8_t* w_scales;
  Epi ep;
  int64_t M, N, K, P;
};
size_t mx_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int parts, const DeviceCaps& caps);
hipError_t launch_mx_grad(const MxGradArgs& a, const DeviceCaps& caps, void* ws, size_t ws_bytes, hipStream_t st);

// Column sums of X [M][N] (mx_sum.hip), to the one row of ep.
size_t mx_sum_workspace_bytes(int64_t M, int64_t N, const DeviceCaps& caps);
hipError_t launch_mx_sum(const void* X, int dt, int64_t M, int64_t N, int64_t ld, const Epi& ep, const DeviceCaps& caps, void* ws,
                         hipStream_t st);

// A layer of experts (mx_moe.hip) for T <= kMoeTokens tokens: x [T][mx_parts(dt)][ldx] bf16 parts
// (rows 16-byte aligned), Hx columns of each (a multiple of 64) to read.
constexpr int kMoeTokens = 64, kMoeTop = 16, kMoeExperts = 512;
constexpr int kMoeParts = 3;  // of what lies between the products: all bits of an fp32
struct MoeArgs {
  const uint16_t* x;
  int64_t ldx, Hx;
  const void* logits;
  int ldt;
  int64_t ldl;
  const uint8_t* W1;
  const uint8_t* w1_scales;
  const uint8_t* W2;
  const uint8_t* w2_scales;
  int64_t T, E, H, F;
  int top;
  int renorm;
  int dt;  // of x and the output
  void* out;
  int64_t ldo;
};
size_t moe_workspace_bytes(const MoeArgs& a, const DeviceCaps& caps);
hipError_t launch_moe(const MoeArgs& a, const DeviceCaps& caps, void* ws, hipStream_t st);

// ---- token scores (include/w8a8.h)

struct TokArgs {
  const void* z;
  int dt;
  int64_t M, V, ld;
  const int64_t* targets;
  int64_t ignore;
  float inv_t;  // fp32(1 / temperature)
  int top;
  float *lp, *ent, *stats, *top_lp;
  int64_t* top_ids;
};
size_t tok_ws_bytes(int64_t M, int64_t V, int top, const DeviceCaps& caps);
hipError_t launch_tok(const TokArgs& a, const DeviceCaps& caps, void* ws, hipStream_t st);

struct TokGradArgs {
  const void* z;
  int dt;
  int64_t M, V, ld;
  const int64_t* targets;
  int64_t ignore;
  float inv_t;
  int top;
  const float *stats, *ent;
  const int64_t* top_ids;
  const float *g, *h, *a;
  void* dz;
  int64_t ldd;
};
hipError_t launch_tok_grad(const TokGradArgs& a, const DeviceCaps& caps, hipStream_t st);

}  // namespace w4
