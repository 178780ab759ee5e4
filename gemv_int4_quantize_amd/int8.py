"""PyTorch-facing binding of the 8-bit integer linear operators.

``quantize_int8`` turns rows (tokens, or the output channels of a weight) into int8 codes
with one fp32 scale a row; ``mm_int8`` multiplies two such operands, quantizing float
activations on the way; ``mm_int8_t`` is the product's input gradient on the same weight.
Argument marshalling only: every step runs in the library's gfx950 kernels (see
include/w8a8.h for the contract).
"""

from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import check, lib
from .ops import _ODT, _WDT, _stream


@dataclass
class Int8Rows:
    """Rows of int8 codes with one fp32 scale each: row r stands for codes[r, :cols] * scales[r].

    codes is int8 [rows][pitch], pitch = cols rounded up to a multiple of 64, 16-byte aligned,
    contiguous, with zeros in the columns past ``cols``; scales is a contiguous fp32 [rows].
    A weight W [N][K] has one row (and scale) per output channel, activations X [M][K] one
    per token."""

    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int


def _pitch(cols: int) -> int:
    return (cols + 63) // 64 * 64


def check_device(*tensors) -> int:
    """The index of the one HIP device that the tensors (None among them) are on."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        d = t.device
        if dev is None:
            if d.type != "cuda":
                raise ValueError("tensors must be on a HIP device")
            dev = d
        elif d != dev:
            if d.type != "cuda":
                raise ValueError("tensors must be on a HIP device")
            raise ValueError(f"tensors on {dev} and {d}: one device is wanted")
    return dev.index


class on_device:
    """Device `index` as the current one (launches go to the current device) for a call."""

    __slots__ = ("index", "back")

    def __init__(self, index: int):
        self.index = index

    def __enter__(self):
        now = torch._C._cuda_getDevice()
        self.back = now if now != self.index else None
        if self.back is not None:
            torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        if self.back is not None:
            torch.cuda.set_device(self.back)


def space(nbytes: int, device):
    """A call's workspace (None for none) from torch's allocator, in the current stream's order."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


class _Once(torch.autograd.Function):
    """The identity of a gradient, as a function of what it was computed from: differentiating it
    raises.  (A backward that is marked as once differentiable raises only where the gradient it
    was given requires grad itself; its dependence on the saved tensors would go unnoticed.)"""

    @staticmethod
    def forward(ctx, grad, what, *of):
        ctx.what = what
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.what}: trying to differentiate twice (its gradient has no derivative here)")


def once(grad: torch.Tensor, what: str, *of) -> torch.Tensor:
    """The result `grad` of a backward, computed from the tensors `of` (None among them), marked so
    that a second derivative through it raises."""
    return _Once.apply(grad, what, *of) if torch.is_grad_enabled() else grad


def float_rows(x: torch.Tensor, what: str) -> torch.Tensor:
    """x as the library takes float rows: 2-D, columns next to one another, any row stride."""
    if x.dim() != 2:
        raise ValueError(f"{what} must be a 2-D tensor (got {x.dim()}-D)")
    if x.dtype not in _WDT:
        raise TypeError(f"{what} must be float32, float16 or bfloat16 (got {x.dtype})")
    if (x.shape[1] > 1 and x.stride(1) != 1) or (x.shape[0] > 1 and x.stride(0) < x.shape[1]):
        x = x.contiguous()
    return x


def _row_stride(x: torch.Tensor) -> int:
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _check_rows(w: Int8Rows, what: str) -> None:
    c, s = w.codes, w.scales
    if c.dtype is not torch.int8 or c.shape != (w.rows, _pitch(w.cols)) or not c.is_contiguous():
        raise ValueError(f"{what}: codes must be a contiguous int8 [{w.rows}][{_pitch(w.cols)}] tensor")
    if s.dtype is not torch.float32 or s.numel() != w.rows or not s.is_contiguous():
        raise ValueError(f"{what}: scales must be a contiguous float32 vector of length {w.rows}")


def quantize_int8(x: torch.Tensor) -> Int8Rows:
    """Int8 codes and scales of the rows of x [rows][cols] (float32, float16 or bfloat16; rows may
    be strided): scale = max |x| / 127, code = rint(x / scale).  A row with a NaN or an infinity
    gets a NaN scale."""
    x = float_rows(x, "x")
    rows, cols = x.shape
    with on_device(check_device(x)):
        out = Int8Rows(torch.empty((rows, _pitch(cols)), dtype=torch.int8, device=x.device),
                       torch.empty(rows, dtype=torch.float32, device=x.device), rows, cols)
        check(lib().w8_quantize_rows(x.data_ptr(), _WDT[x.dtype], rows, cols, _row_stride(x), out.codes.data_ptr(),
                                     out.scales.data_ptr(), _stream(x.device)))
    return out


_ONE = _lib.W4OutSeg * 1


def _new_output(M: int, width: int, dt: torch.dtype, device):
    """A tensor [M][width] for a result, and its segment."""
    if dt not in _ODT:
        raise ValueError(f"outputs must be float32, float16 or bfloat16 (got {dt})")
    out = torch.empty((M, width), dtype=dt, device=device)
    return out, _ONE((out.data_ptr(), width, width))


def _segments(outs, M: int, width: int, dt: torch.dtype):
    if dt not in _ODT:
        raise ValueError(f"outputs must be float32, float16 or bfloat16 (got {dt})")
    segs = (_lib.W4OutSeg * len(outs))()
    cols = 0
    for i, o in enumerate(outs):
        if o.dtype != dt or o.dim() != 2 or o.shape[0] != M or (o.shape[1] > 1 and o.stride(1) != 1):
            raise ValueError(f"each output must be a 2-D [{M}][cols] {dt} tensor with contiguous rows")
        n = o.shape[1]
        cols += n
        segs[i] = _lib.W4OutSeg(o.data_ptr(), n, o.stride(0) if M > 1 else n)
    if cols != width:
        raise ValueError(f"the outputs' columns must sum to {width}")
    return segs


# workspace sizes depend on the sizes alone
@functools.lru_cache(maxsize=4096)
def _product_bytes(M: int, N: int, K: int, x_dtype: int) -> int:
    size = ctypes.c_size_t(0)
    check(lib().w8a8_workspace_bytes(M, N, K, x_dtype, ctypes.byref(size)))
    return size.value


@functools.lru_cache(maxsize=4096)
def _gradient_bytes(M: int, N: int, K: int, ld: int) -> int:
    size = ctypes.c_size_t(0)
    check(lib().w8a16_mm_t_workspace_bytes(M, N, K, ld, ctypes.byref(size)))
    return size.value


def _product(a, w: Int8Rows, bias, outs, dt: torch.dtype, segs=None):
    """One product written to `outs`, which cover its columns in order (segs: theirs, if made)."""
    N, K = w.rows, w.cols
    _check_rows(w, "weight")
    if bias is not None and (bias.dtype != dt or bias.numel() != N or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous {dt} vector of length {N}")
    ready = isinstance(a, Int8Rows)
    if ready:
        _check_rows(a, "activations")
        M, width, x, xs, xdt = a.rows, a.cols, a.codes, a.scales, -1
    else:
        M, width = a.shape
        x, xs, xdt = a, None, _WDT[a.dtype]
    if width != K:
        raise ValueError(f"activation width {width} does not match the weight ({N}x{K})")
    if segs is None:
        segs = _segments(outs, M, N, dt)
    L = lib()
    with on_device(check_device(x, xs, w.codes, w.scales, bias, *outs)):
        size = _product_bytes(M, N, K, xdt)
        ws = space(size, x.device)
        bp = bias.data_ptr() if bias is not None else None
        wp = ws.data_ptr() if ws is not None else None
        if ready:
            status = L.w8a8_mm(x.data_ptr(), xs.data_ptr(), M, w.codes.data_ptr(), w.scales.data_ptr(), N, K, bp,
                               _ODT[dt], segs, len(outs), wp, size, _stream(x.device))
        else:
            status = L.w8a8_linear(x.data_ptr(), xdt, _row_stride(x), M, w.codes.data_ptr(), w.scales.data_ptr(), N, K,
                                   bp, _ODT[dt], segs, len(outs), wp, size, _stream(x.device))
    check(status)


def mm_int8(a, w: Int8Rows, bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
            out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Y = A @ W^T (+ bias) in 8-bit integers, one scale per token and one per channel.

    `a` is a float tensor [M][K] (float32, float16 or bfloat16), quantized per token within the
    call, or an Int8Rows.  The integer sums are exact; each is scaled and the bias added in
    fp32, then rounded once to the output dtype: fp32 unless `out_dtype` (or `out`) asks for
    bfloat16 / float16.  The bias has the output dtype."""
    if not isinstance(a, Int8Rows):
        a = float_rows(a, "activations")
    dev = w.codes.device
    M = a.rows if isinstance(a, Int8Rows) else a.shape[0]
    dt = out_dtype if out_dtype is not None else (out.dtype if out is not None else torch.float32)
    segs = None
    if out is None:
        out, segs = _new_output(M, w.rows, dt, dev)
    elif out.shape != (M, w.rows) or out.dtype != dt:
        raise ValueError(f"out must be a {dt} tensor of shape ({M}, {w.rows})")
    _product(a, w, bias, (out,), dt, segs)
    return out


def mm_int8_split(a, w: Int8Rows, outs: list[torch.Tensor], bias: torch.Tensor | None = None) -> list[torch.Tensor]:
    """mm_int8 written to separate outputs in one launch: outs[i] [M][n_i] receives the next n_i
    output columns (for a fused Q/K/V weight: Q, K and V).  At most four outputs, of one dtype;
    they may be row-strided views.  The bias, if any, spans all output columns in that dtype."""
    if not isinstance(a, Int8Rows):
        a = float_rows(a, "activations")
    if not outs:
        raise ValueError("at least one output is wanted")
    _product(a, w, bias, list(outs), outs[0].dtype)
    return list(outs)


def mm_int8_t(dy: torch.Tensor, w: Int8Rows, out: torch.Tensor | None = None,
              out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """dX = dY @ W, the input gradient of ``mm_int8``, on the same int8 weight.

    dY [M][N] is bfloat16 or float16 (rows may be strided); the weight operand is codes * scale
    rounded to that dtype (float16: to its precision, whatever the size of the scales), sums are
    fp32 and the result is rounded once to `out_dtype` (fp32 unless given)."""
    if dy.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"dY must be bfloat16 or float16 (got {dy.dtype})")
    dy = float_rows(dy, "dY")
    M, width = dy.shape
    N, K = w.rows, w.cols
    if width != N:
        raise ValueError(f"gradient width {width} does not match the weight ({N}x{K})")
    _check_rows(w, "weight")
    dt = out_dtype if out_dtype is not None else (out.dtype if out is not None else torch.float32)
    if out is None:
        out, segs = _new_output(M, K, dt, dy.device)
    elif out.shape != (M, K) or out.dtype != dt:
        raise ValueError(f"out must be a {dt} tensor of shape ({M}, {K})")
    else:
        segs = _segments((out,), M, K, dt)
    ld = _row_stride(dy)
    with on_device(check_device(dy, w.codes, w.scales, out)):
        size = _gradient_bytes(M, N, K, ld if dy.data_ptr() % 16 == 0 else -1)
        ws = space(size, dy.device)
        status = lib().w8a16_mm_t(dy.data_ptr(), _WDT[dy.dtype], ld, M, w.codes.data_ptr(), w.scales.data_ptr(), N, K,
                                  _ODT[dt], segs, 1, ws.data_ptr() if ws is not None else None, size,
                                  _stream(dy.device))
    check(status)
    return out


@functools.lru_cache(maxsize=4096)
def _gradient32_bytes(M: int, N: int, K: int) -> int:
    size = ctypes.c_size_t(0)
    check(lib().w8a32_mm_t_workspace_bytes(M, N, K, ctypes.byref(size)))
    return size.value


def gradient_of_fp32(dy: torch.Tensor, w: Int8Rows, out_dtype: torch.dtype) -> torch.Tensor:
    """mm_int8_t of an fp32 dY [M][N] with fp16 operands: each of its rows enters at a power of two of
    its own, so that no size of dY is lost."""
    dy = float_rows(dy, "dY")
    M, N, K = dy.shape[0], w.rows, w.cols
    if dy.dtype is not torch.float32 or dy.shape[1] != N:
        raise ValueError(f"dY must be a float32 tensor of width {N}")
    _check_rows(w, "weight")
    out, segs = _new_output(M, K, out_dtype, dy.device)
    with on_device(check_device(dy, w.codes, w.scales)):
        size = _gradient32_bytes(M, N, K)
        ws = space(size, dy.device)
        status = lib().w8a32_mm_t(dy.data_ptr(), _row_stride(dy), M, w.codes.data_ptr(), w.scales.data_ptr(), N, K,
                                  _ODT[out_dtype], segs, 1, ws.data_ptr() if ws is not None else None, size,
                                  _stream(dy.device))
    check(status)
    return out


def int8_kernel_for(M: int, N: int, K: int) -> str | None:
    """Name of the kernel that multiplies M float tokens by a weight of this shape (host-side query)."""
    r = lib().w8a8_kernel(M, N, K, _lib.DT_BF16)
    return r.decode() if r is not None else None
