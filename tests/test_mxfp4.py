"""The microscaled 4-bit operators: refusals on the host, and on the GPU the quantizer bit for bit,
the product and its gradient exactly where sums are exact and against 64 bits elsewhere."""

import ctypes

import numpy as np
import pytest
import torch

import gemv_int4_quantize_amd as w4
from gemv_int4_quantize_amd import _lib

DEV = "cuda:0"
EPS32 = 2.0**-24  # half an ulp of 1 in fp32
HALF_ULP = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float32: 2.0**-149, torch.float16: 2.0**-24, torch.bfloat16: 2.0**-133}
MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
FLOATS = [torch.float32, torch.float16, torch.bfloat16]


# ---------------------------------------------------------------- host only


def _p(v=0x10000):  # an aligned address that is never dereferenced: every call below is refused
    return ctypes.c_void_p(v)


def _seg(cols, y=0x10000, ld=None):
    s = (_lib.W4OutSeg * 1)()
    s[0].Y, s[0].cols, s[0].ld = y, cols, cols if ld is None else ld
    return s


def test_header_and_exports():
    import os
    import re

    path = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "mxfp4.h")
    names = re.findall(r"^(?:int|int64_t|const char\*)\s+(mx4\w+)\s*\(", open(path).read(), flags=re.M)
    assert sorted(names) == sorted(_lib.EXPORTS_MX)
    for n in names:
        assert hasattr(w4.lib(), n), n


def test_pitch():
    L = w4.lib()
    assert [L.mx4_pitch(k) for k in (-3, 0, 1, 128, 129, 11008)] == [-1, -1, 128, 128, 256, 11008]


def test_quantize_refusals():
    q = w4.lib().mx4_quantize_rows
    assert q(_p(), 0, 4, 0, 64, _p(), _p(), None) == _lib.W4_ERR_INVALID
    assert q(_p(), 7, 4, 64, 64, _p(), _p(), None) == _lib.W4_ERR_INVALID
    assert q(_p(), 2, -1, 64, 64, _p(), _p(), None) == _lib.W4_ERR_INVALID
    assert q(_p(), 2, 4, 64, 63, _p(), _p(), None) == _lib.W4_ERR_INVALID
    assert q(None, 2, 4, 64, 64, _p(), _p(), None) == _lib.W4_ERR_INVALID
    assert q(_p(), 2, 4, 64, 64, None, _p(), None) == _lib.W4_ERR_INVALID
    assert q(_p(), 2, 4, 64, 64, _p(), None, None) == _lib.W4_ERR_INVALID
    assert q(_p(), 2, 4, 1 << 22, 1 << 22, _p(), _p(), None) == _lib.W4_ERR_UNSUPPORTED
    assert q(_p(), 2, 1 << 30, 64, 64, _p(), _p(), None) == _lib.W4_ERR_UNSUPPORTED
    assert q(_p(0x10001), 2, 4, 64, 64, _p(), _p(), None) == _lib.W4_ERR_ALIGN
    assert q(_p(), 2, 4, 64, 64, _p(0x10008), _p(), None) == _lib.W4_ERR_ALIGN
    assert q(_p(), 2, 4, 64, 64, _p(), _p(0x10002), None) == _lib.W4_ERR_ALIGN
    assert q(None, 2, 0, 64, 64, None, None, None) == _lib.W4_OK
    d = w4.lib().mx4_dequantize_rows
    assert d(_p(), _p(), 4, 64, _p(), 5, 64, None) == _lib.W4_ERR_INVALID
    assert d(_p(), _p(), 4, 64, None, 0, 64, None) == _lib.W4_ERR_INVALID
    assert d(None, _p(), 4, 64, _p(), 0, 64, None) == _lib.W4_ERR_INVALID
    assert d(_p(), _p(), 4, 64, _p(), 0, 63, None) == _lib.W4_ERR_INVALID
    assert d(_p(), _p(), 4, 64, _p(0x10002), 0, 64, None) == _lib.W4_ERR_ALIGN
    assert d(None, None, 0, 64, None, 0, 64, None) == _lib.W4_OK


def test_product_refusals():
    def mm(A=_p(), sa=_p(), M=4, W=_p(), sw=_p(), N=64, K=128, bias=None, dt=0, segs=_seg(64), n=1, ws=None, wsb=0):
        return w4.lib().mx4_mm(A, sa, M, W, sw, N, K, bias, dt, segs, n, ws, wsb, None)

    assert mm(M=-1) == _lib.W4_ERR_INVALID
    assert mm(N=0) == _lib.W4_ERR_INVALID
    assert mm(K=0) == _lib.W4_ERR_INVALID
    assert mm(K=1 << 22) == _lib.W4_ERR_UNSUPPORTED
    assert mm(A=None) == _lib.W4_ERR_INVALID
    assert mm(sw=None) == _lib.W4_ERR_INVALID
    assert mm(W=_p(0x10004)) == _lib.W4_ERR_ALIGN
    assert mm(sa=_p(0x10001)) == _lib.W4_ERR_ALIGN
    assert mm(dt=3) == _lib.W4_ERR_INVALID
    assert mm(segs=_seg(63)) == _lib.W4_ERR_INVALID
    assert mm(segs=_seg(64, ld=60)) == _lib.W4_ERR_INVALID
    assert mm(segs=_seg(64, y=None)) == _lib.W4_ERR_INVALID
    assert mm(n=5) == _lib.W4_ERR_INVALID
    assert mm(bias=_p(0x10002)) == _lib.W4_ERR_ALIGN
    assert mm(ws=_p(0x10004), wsb=64) == _lib.W4_ERR_ALIGN
    assert mm(M=0, A=None) == _lib.W4_OK

    L = w4.lib()

    def linear(X=_p(), dt=2, ld=128, M=64, ws=None, wsb=0):
        return L.mx4_linear(X, dt, ld, M, _p(), _p(), 64, 128, None, 0, _seg(64), 1, ws, wsb, None)

    assert linear(dt=5) == _lib.W4_ERR_INVALID
    assert linear(ld=100) == _lib.W4_ERR_INVALID
    assert linear(X=None) == _lib.W4_ERR_INVALID
    size = ctypes.c_size_t(0)
    assert L.mx4_workspace_bytes(64, 64, 128, 2, ctypes.byref(size)) == 0 and size.value >= 64 * 64 + 64 * 4
    assert linear() == _lib.W4_ERR_RESOURCE
    assert linear(ws=_p(), wsb=size.value - 1) == _lib.W4_ERR_RESOURCE
    assert L.mx4_workspace_bytes(64, 64, 128, 9, ctypes.byref(size)) == _lib.W4_ERR_INVALID
    assert L.mx4_workspace_bytes(64, 64, 128, 2, None) == _lib.W4_ERR_INVALID


def test_gradient_refusals():
    L = w4.lib()

    def mt(dY=_p(), dt=2, ld=64, M=4, N=64, K=128, segs=_seg(128), ws=None, wsb=0):
        return L.mx4_mm_t(dY, dt, ld, M, _p(), _p(), N, K, 0, segs, 1, ws, wsb, None)

    assert mt(dt=4) == _lib.W4_ERR_INVALID
    assert mt(dY=None) == _lib.W4_ERR_INVALID
    assert mt(ld=63) == _lib.W4_ERR_INVALID
    assert mt(segs=_seg(64)) == _lib.W4_ERR_INVALID
    assert mt(N=1 << 20, ld=1 << 20) == _lib.W4_ERR_UNSUPPORTED
    assert mt(N=63) == _lib.W4_ERR_RESOURCE  # an unaligned dY needs its copy
    assert mt(dY=_p(0x10002)) == _lib.W4_ERR_RESOURCE
    assert mt(dt=0) == _lib.W4_ERR_RESOURCE and mt(dt=1) == _lib.W4_ERR_RESOURCE  # their parts
    assert mt(M=0, dY=None) == _lib.W4_OK
    # the reported workspace is what the call asks for
    size = ctypes.c_size_t(0)
    for M, N, dt, ld in ((4, 64, 2, 1 << 22), (4, 64, 2, 64), (4, 60, 2, 60), (4, 64, 2, -1), (1, 64, 2, 67), (4, 64, 1, 64),
                         (4, 63, 0, 63), (2, 64, 2, 68)):
        assert L.mx4_mm_t_workspace_bytes(M, N, 128, dt, ld, ctypes.byref(size)) == 0
        copied = dt != 2 or N % 8 != 0 or (ld % 8 != 0 or ld >= 1 << 22 if M > 1 else False) or ld < 0
        bytes_ = M * 64 * 2 * (3 if dt == 0 else 2 if dt == 1 else 1)
        assert (size.value >= bytes_) == copied, (M, N, dt, ld)
        if copied and ld > 0:
            assert mt(dt=dt, ld=ld, M=M, N=N, ws=_p(), wsb=bytes_ - 1) == _lib.W4_ERR_RESOURCE, (M, N, dt, ld)


def test_binding_refusals():
    w = w4.MXFP4Rows(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 4, dtype=torch.uint8), 8, 64)
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="HIP device"):
        w4.mm_mxfp4(x, w)
    with pytest.raises(ValueError, match="HIP device"):
        w4.quantize_mxfp4(x)
    with pytest.raises(ValueError, match="width"):
        w4.mm_mxfp4(torch.zeros(2, 63), w)
    with pytest.raises(TypeError):
        w4.mm_mxfp4(torch.zeros(2, 64, dtype=torch.float64), w)
    with pytest.raises(ValueError, match="bias"):
        w4.mm_mxfp4(x, w, bias=torch.zeros(7))
    with pytest.raises(ValueError, match="out must"):
        w4.mm_mxfp4(x, w, out=torch.zeros(2, 9))
    with pytest.raises(ValueError, match="codes"):
        w4.mm_mxfp4(x, w4.MXFP4Rows(torch.zeros(8, 32, dtype=torch.uint8), w.scales, 8, 64))
    with pytest.raises(ValueError, match="scales"):
        w4.mm_mxfp4(x, w4.MXFP4Rows(w.codes, torch.zeros(8, 2, dtype=torch.uint8), 8, 64))
    with pytest.raises(ValueError, match="at least one output"):
        w4.mm_mxfp4_split(x, w, [])
    with pytest.raises(ValueError, match="sum to"):
        w4.mm_mxfp4_split(x, w, [torch.zeros(2, 3)])
    with pytest.raises(TypeError):
        w4.mm_mxfp4_t(torch.zeros(2, 8, dtype=torch.int32), w)
    with pytest.raises(ValueError, match="width"):
        w4.mm_mxfp4_t(torch.zeros(2, 9, dtype=torch.bfloat16), w)
    with pytest.raises(ValueError, match="outputs must"):
        w4.dequantize_mxfp4(w, torch.int8)
    with pytest.raises(ValueError, match="out_dtype"):
        w4.MXFP4Linear(w, out_dtype=torch.int8)


def test_sum_refusals():
    L, size = w4.lib(), ctypes.c_size_t(0)
    f32 = _lib.DT_F32

    def call(dtype=f32, M=4, N=8, ld=8, x=_p(), out=_p(), out_dtype=f32, ws=None, ws_bytes=0):
        return L.mx4_sum_rows(x, dtype, M, N, ld, out, out_dtype, ws, ws_bytes, None)

    for bad in (dict(dtype=7), dict(M=-1), dict(N=0), dict(ld=7), dict(x=None), dict(out=None), dict(out_dtype=9)):
        assert call(**bad) == _lib.W4_ERR_INVALID, bad
    assert call(N=1 << 30, ld=1 << 30) == _lib.W4_ERR_UNSUPPORTED
    for bad in (dict(x=_p(0x10002)), dict(out=_p(0x10001)), dict(ws=_p(0x10008), ws_bytes=64)):
        assert call(**bad) == _lib.W4_ERR_ALIGN, bad
    assert L.mx4_sum_workspace_bytes(4096, 8, ctypes.byref(size)) == 0 and size.value > 0
    assert call(M=4096) == _lib.W4_ERR_RESOURCE and call(M=4096, ws=_p(), ws_bytes=size.value - 1) == _lib.W4_ERR_RESOURCE
    assert L.mx4_sum_workspace_bytes(4, 8, None) == _lib.W4_ERR_INVALID
    with pytest.raises(ValueError, match="HIP device"):
        w4.mxfp4.sum_rows(torch.zeros(2, 3))
    with pytest.raises(ValueError, match="outputs must"):
        w4.mxfp4.sum_rows(torch.zeros(2, 3), torch.int8)
    with pytest.raises(TypeError):
        w4.mxfp4.sum_rows(torch.zeros(2, 3, dtype=torch.int32))


def test_kernel_names():
    k = w4.lib().mx4_kernel
    assert k(2, 4096, 4096, -1) == b"mx4_decode" and k(2, 4096, 4096, _lib.DT_BF16) == b"mx4_decode_fused"
    assert k(32, 4096, 4096, -1) == k(32, 4096, 4096, _lib.DT_BF16) == b"mx4_few"
    assert k(64, 4096, 4096, -1) == k(64, 4096, 4096, _lib.DT_F32) is not None
    assert w4.mxfp4_kernel_for(8192, 8192, 8192) == "mx4_256x256"
    for bad in ((2, 4096, 4096, 9), (0, 64, 64, -1), (4, 0, 64, -1), (4, 64, 1 << 22, -1)):
        assert k(*bad) is None


def test_second_derivatives_raise(monkeypatch):
    """The layer's gradient is no function that autograd knows.  (The launches are replaced by torch on
    the CPU: what is left is the autograd.)"""
    from gemv_int4_quantize_amd import mxfp4

    weight = torch.randn(8, 64)
    monkeypatch.setattr(mxfp4, "mm_mxfp4", lambda x, w, bias=None, out_dtype=None: (x.float() @ weight.t()).to(out_dtype))
    seen = []

    def back(g, w, out_dtype=torch.float32):
        seen.append(g.dtype)
        return (g.float() @ weight).to(out_dtype)

    monkeypatch.setattr(mxfp4, "mm_mxfp4_t", back)
    monkeypatch.setattr(mxfp4, "sum_rows", lambda g, out_dtype: g.float().sum(0).to(out_dtype))
    w = w4.MXFP4Rows(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 4, dtype=torch.uint8), 8, 64)
    bias = torch.zeros(8, requires_grad=True)
    for b in (None, bias):
        x = torch.randn(3, 64, requires_grad=True)
        (g,) = torch.autograd.grad(w4.mxfp4_linear(x, w, b).square().sum() + (x**3).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="twice|once_differentiable"):
            g.square().sum().backward()
    # the types that dY enters in
    for xd, od, want in ((torch.bfloat16, None, torch.bfloat16), (torch.float32, None, torch.float32),
                         (torch.float16, None, torch.float32), (torch.float32, torch.bfloat16, torch.bfloat16)):
        x = torch.randn(3, 64).to(xd).requires_grad_()
        w4.mxfp4_linear(x, w, out_dtype=od).sum().backward()
        assert seen[-1] == want and x.grad.dtype == xd


# ---------------------------------------------------------------- GPU


def _values(codes, scales, cols):
    """The values of codes [rows][P/2] and scales [rows][P/32] in 64 bits."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[0], -1)
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    return (v * np.exp2(scales.astype(np.float64) - 127.0).repeat(32, axis=1))[:, :cols]


def _quantize_ref(x):
    """Codes [rows][P] and scales of rows x (64 bits), step by step from the definition."""
    rows, cols = x.shape
    p = (cols + 127) // 128 * 128
    wide = np.zeros((rows, p))
    wide[:, :cols] = x
    blocks = wide.reshape(rows, -1, 32)
    with np.errstate(invalid="ignore"):
        top = np.abs(blocks).max(axis=2)
    bad = ~np.isfinite(blocks).all(axis=2)
    top = np.where(bad, 1.0, top)
    exp = np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] - 1 - 2 + 127, 0)
    scales = np.where(bad, 255, np.maximum(exp, 0)).astype(np.uint8)
    mag = np.where(bad[:, :, None], 0.0, np.abs(np.where(np.isfinite(blocks), blocks, 0.0)) *
                   np.exp2(127.0 - np.where(bad, 127, scales).astype(np.float64))[:, :, None])
    # the nearest magnitude, of two equally near the one with an even code
    dist = np.abs(mag[..., None] - MAGNITUDES)
    near = dist.min(axis=-1, keepdims=True) == dist
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    sign = np.signbit(np.where(bad[:, :, None], 0.0, blocks))
    return (code + 8 * sign).reshape(rows, p).astype(np.uint8), scales


def _packed(codes):
    return codes[:, 0::2] | codes[:, 1::2] << 4


def _rows(seed, rows, cols, dtype, pad=0, scale=1.0):
    """Seeded rows with per-row magnitudes, as (device tensor of rows `pad` longer, 64-bit numpy)."""
    g = np.random.default_rng(seed)
    a = g.standard_normal((rows, cols)) * np.exp(g.standard_normal((rows, 1))) * scale
    t = torch.from_numpy(a.astype(np.float32)).to(dtype)
    wide = torch.full((rows, cols + pad), float("nan"), dtype=dtype)
    wide[:, :cols] = t
    return wide.to(DEV)[:, :cols], t.double().numpy()


def _weight(seed, n, k, spread=12):
    """A weight of random codes and exponents: (rows on the device, values in 64 bits)."""
    g = np.random.default_rng(seed)
    p = (k + 127) // 128 * 128
    codes = np.zeros((n, p), dtype=np.uint8)
    codes[:, :k] = g.integers(0, 16, (n, k))
    scales = g.integers(120 - spread // 2, 121 + spread // 2, (n, p // 32)).astype(np.uint8)
    w = w4.MXFP4Rows(torch.from_numpy(_packed(codes)).to(DEV), torch.from_numpy(scales).to(DEV), n, k)
    return w, _values(_packed(codes), scales, k)


def _check_rounded(y, ref, size, dtype, what, steps):
    """|y - ref| <= `steps` fp32 roundings of magnitude `size`, and one rounding to dtype."""
    y = y.double().cpu().numpy()
    tol = steps * EPS32 * size + (HALF_ULP[dtype] * (np.abs(ref) + steps * EPS32 * size) + TINY[dtype]
                                  if dtype != torch.float32 else 2.0**-149)
    bad = ~(np.abs(y - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {np.abs(y - ref)[bad].max():.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 7, 1), (5, 64, 0), (2, 129, 3), (9, 2048, 0), (4, 2049, 5),
                                           (33, 31, 0), (7, 11008, 0), (2, 16385, 0), (1, 70001, 2), (300, 96, 8)])
def test_quantize_bits(dtype, rows, cols, pad):
    x, x64 = _rows(rows * 1000 + cols, rows, cols, dtype, pad)
    r = w4.quantize_mxfp4(x)
    codes, scales = _quantize_ref(x64)
    np.testing.assert_array_equal(r.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(r.codes.cpu().numpy(), _packed(codes))
    for out in FLOATS:
        got = w4.dequantize_mxfp4(r, out)
        want = torch.from_numpy(_values(_packed(codes), scales, cols)).to(out)
        assert got.shape == (rows, cols) and torch.equal(got.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
def test_quantize_special_blocks(dtype):
    """Zeros of both signs, subnormals, the largest values, ties, NaN and infinities: a block each."""
    tiny = {torch.float32: 2.0**-149, torch.float16: 2.0**-24, torch.bfloat16: 2.0**-133}[dtype]
    x = np.random.default_rng(3).standard_normal((3, 32 * 12))
    b = x.reshape(3, 12, 32)
    b[:, 0] = 0
    b[:, 1] = -0.0
    b[:, 2] = tiny * np.arange(32)
    b[:, 3] = torch.finfo(dtype).max
    b[:, 4] = torch.finfo(dtype).tiny * 3
    b[:, 5, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5, -0.25, -0.75, -1.25, -2.5, -5.0, 4.0]
    b[:, 6] = b[:, 5] * 2.0**-12
    b[1, 7, 3] = np.nan
    b[1, 8, 31] = np.inf
    b[2, 9, 0] = -np.inf
    b[:, 10] = 0
    b[:, 10, 5] = -tiny
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    r = w4.quantize_mxfp4(t.to(DEV))
    codes, scales = _quantize_ref(t.double().numpy())
    np.testing.assert_array_equal(r.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(r.codes.cpu().numpy(), _packed(codes))
    back = w4.dequantize_mxfp4(r, torch.float32).cpu().numpy().reshape(3, 12, 32)
    bad = np.zeros((3, 12), bool)
    bad[1, 7] = bad[1, 8] = bad[2, 9] = True
    assert (np.isnan(back).all(axis=2) == bad).all() and np.isfinite(back[~bad]).all()
    w, _ = _weight(1, 24, 384)
    for rep in (1, 20):  # few tokens, and a tile of them
        y = w4.mm_mxfp4(t.to(DEV).repeat(rep, 1), w).cpu().numpy()
        assert np.isnan(y[1::3]).all() and np.isnan(y[2::3]).all()
        # fp32's and bf16's largest, quantized to 6 * 2^125, times weights up to 6 * 2^-1 pass 2^128
        if dtype == torch.float16:
            assert np.isfinite(y[0::3]).all()


@pytest.mark.gpu
def test_all_codes_and_scales():
    """Every byte of codes at every scale, to each type."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    w = w4.MXFP4Rows(codes.to(DEV), scales.to(DEV), 256, 512)
    want = _values(codes.numpy(), scales.numpy(), 512)
    want[255] = np.nan
    for dtype in FLOATS:
        ref = torch.from_numpy(want).to(dtype)
        got = w4.dequantize_mxfp4(w, dtype).cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(got[:255], ref[:255])


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 2048, 2048), (2, 33, 70), (3, 1000, 4096), (4, 512, 11008), (5, 100, 129),
          (16, 48, 4096), (17, 515, 2048), (32, 256, 1030), (33, 130, 640), (64, 96, 8192), (65, 300, 1000),
          (127, 257, 511), (128, 128, 128), (200, 640, 192), (257, 259, 300), (300, 1003, 1555), (515, 2050, 257),
          (8, 5000, 300), (12, 9000, 384), (4, 9000, 257), (700, 2304, 640),
          (16, 8000, 300), (29, 8190, 1100), (24, 16384, 640), (32, 9000, 256), (1, 40, 60000), (6, 8, 5000), (31, 17, 60)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", FLOATS)
def test_product(m, n, k, dtype):
    """Float activations and rows quantized before give the same sums, near those in 64 bits."""
    x, x64 = _rows(m + n + k, m, k, dtype, pad=3 if m % 2 else 0)
    w, w64 = _weight(n + k, n, k)
    bias = torch.from_numpy(np.random.default_rng(5).standard_normal(n).astype(np.float32)).to(dtype)
    codes, scales = _quantize_ref(x64)
    a64 = _values(_packed(codes), scales, k)
    ref, size = a64 @ w64.T, np.abs(a64) @ np.abs(w64).T
    b = bias.double().numpy()
    xq = w4.quantize_mxfp4(x)
    # exact products; k sums in any order, each rounded or cut (2 EPS32), and the bias
    for a in (x, xq):
        y = w4.mm_mxfp4(a, w, bias=bias.to(DEV), out_dtype=dtype)
        _check_rounded(y, ref + b, size + np.abs(b), dtype, f"{m}x{n}x{k}", steps=2 * k + 4)
        assert torch.equal(w4.mm_mxfp4(a, w, bias=bias.to(DEV), out_dtype=dtype), y)  # the same bits again
    _check_rounded(w4.mm_mxfp4(x, w), ref, size, torch.float32, f"{m}x{n}x{k} fp32", steps=2 * k + 4)


EXACT = SHAPES + [(40, 4200, 6400), (1500, 1300, 1030), (700, 23000, 256), (2, 40, 70001), (20, 24, 70001)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", EXACT)
def test_product_whole_numbers(m, n, k):
    """Codes at one power: sums of multiples of 1/4 below 36 k < 2^22, exact in any order."""
    assert 36 * k < 1 << 22
    g = torch.Generator(device=DEV).manual_seed(m * 7 + n)

    def rows(r):
        c = torch.randint(0, 256, (r, (k + 127) // 128 * 64), dtype=torch.uint8, device=DEV, generator=g)
        c[:, (k + 1) // 2:] = 0
        if k % 2:
            c[:, k // 2] &= 15
        return w4.MXFP4Rows(c, torch.full((r, (k + 127) // 128 * 4), 127, dtype=torch.uint8, device=DEV), r, k)

    a, w = rows(m), rows(n)
    y = w4.mm_mxfp4(a, w)
    ref = w4.dequantize_mxfp4(a, torch.float32).double() @ w4.dequantize_mxfp4(w, torch.float32).double().t()
    assert torch.equal(y.double(), ref)
    if m <= 4:  # the same tokens as floats: blocks whose largest magnitude is 6 or 4 keep the power
        x = w4.dequantize_mxfp4(a, torch.float32)
        x[:, ::32] = 6.0
        xq = w4.quantize_mxfp4(x)
        assert torch.equal(w4.dequantize_mxfp4(xq, torch.float32), x)
        assert torch.equal(w4.mm_mxfp4(x, w), w4.mm_mxfp4(xq, w))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 3, 9, 20, 70, 300])
@pytest.mark.parametrize("k", [32, 128, 129, 256, 384, 640, 1000])
def test_product_every_block(m, k):
    """One block of one row at a time: its exponent meets its codes, wherever it lies in a stage."""
    n = 40
    w, w64 = _weight(k, n, k, spread=60)
    blocks = (k + 31) // 32
    for at in range(0, blocks, max(1, blocks // 9)):
        x = torch.zeros(m, k, device=DEV)
        powers = torch.arange(m) % 40 - 20
        x[:, at * 32] = torch.from_numpy(np.exp2(powers.numpy().astype(np.float32))).to(DEV)
        y = w4.mm_mxfp4(x, w).double().cpu().numpy()
        ref = np.exp2(powers.numpy().astype(np.float64))[:, None] * w64[:, at * 32][None]
        assert (y == ref).all(), at


@pytest.mark.gpu
def test_product_of_any_power():
    """The least and largest powers on either side, products in and out of fp32's range."""
    for m in (2, 12, 40):
        for ea, ew in ((0, 254), (254, 0), (40, 200), (0, 120), (127, 0), (10, 110)):
            a, _ = _weight(m, m, 256)
            w, _ = _weight(9, 24, 256)
            a.scales.fill_(ea)
            w.scales.fill_(ew)
            y = w4.mm_mxfp4(a, w).double()
            a.scales.fill_(127)
            w.scales.fill_(127)
            want = w4.mm_mxfp4(a, w).double() * 2.0 ** (ea + ew - 254)
            assert torch.equal(y, want.float().double()), (m, ea, ew)


@pytest.mark.gpu
def test_product_nan_blocks():
    """A NaN block of the weight reaches its channel alone, past-the-end blocks none."""
    for m in (1, 4, 10, 40, 200):
        for k in (128, 300, 640):
            w, _ = _weight(2, 50, k)
            x = torch.randn(m, k, device=DEV)
            want = w4.mm_mxfp4(x, w)
            w.scales[17, (k - 1) // 32] = 255
            y = w4.mm_mxfp4(x, w)
            assert torch.isnan(y[:, 17]).all()
            y[:, 17] = want[:, 17]
            assert torch.equal(y, want)
            x[0, 5] = float("nan")
            y = w4.mm_mxfp4(x, w)
            assert torch.isnan(y[0]).all() and torch.isfinite(y[1:, :17]).all()


@pytest.mark.gpu
def test_product_split_outputs_and_views():
    m, k = 37, 320
    w, _ = _weight(8, 24 + 8 + 9, k)
    x, _ = _rows(4, m, k, torch.bfloat16)
    whole = w4.mm_mxfp4(x, w, out_dtype=torch.bfloat16)
    bufs = [torch.full((m, c + 5), 7.0, dtype=torch.bfloat16, device=DEV) for c in (24, 8, 9)]
    w4.mm_mxfp4_split(x, w, [b[:, 2:-3] for b in bufs])
    assert torch.equal(torch.cat([b[:, 2:-3] for b in bufs], 1), whole)
    for b in bufs:
        assert (b[:, :2] == 7).all() and (b[:, -3:] == 7).all()
    for mm in (1, 4, 12, 40):  # rows before and after the output stay as they are
        x, _ = _rows(mm, mm, k, torch.bfloat16)
        guard = torch.full((mm + 2, 41), 3.0, device=DEV)
        w4.mm_mxfp4(x, w, out=guard[1:-1])
        assert (guard[0] == 3).all() and (guard[-1] == 3).all() and (guard[1:-1] != 3).any()


@pytest.mark.gpu
def test_slices_of_rows():
    """Channels of a fused weight, and an aligned part of a buffer: rows are rows wherever they lie."""
    w, _ = _weight(3, 96, 200)
    x = torch.randn(5, 200, device=DEV)
    y = w4.mm_mxfp4(x, w)
    part = w4.MXFP4Rows(w.codes[33:70], w.scales[33:70], 37, 200)
    assert torch.equal(w4.mm_mxfp4(x, part), y[:, 33:70])
    dy = torch.randn(7, 37, device=DEV).bfloat16()
    whole = torch.zeros(7, 96, device=DEV).bfloat16()
    whole[:, 33:70] = dy
    assert torch.equal(w4.mm_mxfp4_t(dy, part), w4.mm_mxfp4_t(dy.contiguous(), part))
    torch.testing.assert_close(w4.mm_mxfp4_t(dy, part), w4.mm_mxfp4_t(whole, w), rtol=1e-5, atol=1e-5)


@pytest.mark.gpu
def test_no_rows():
    w, _ = _weight(2, 8, 64)
    for dtype in FLOATS:
        x = torch.empty(0, 64, dtype=dtype, device=DEV)
        assert w4.mm_mxfp4(x, w).shape == (0, 8)
        assert w4.mm_mxfp4_t(torch.empty(0, 8, dtype=dtype, device=DEV), w).shape == (0, 64)
        q = w4.quantize_mxfp4(x)
        assert q.codes.shape == (0, 64) and w4.dequantize_mxfp4(q).shape == (0, 64) and w4.mm_mxfp4(q, w).shape == (0, 8)


@pytest.mark.gpu
def test_far_offsets():
    """A weight of more than 2^31 bytes, and activations of more than 2^31 elements."""
    n, k = 70003, 65536
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV)
    w = w4.MXFP4Rows(codes, torch.full((n, k // 32), 127, dtype=torch.uint8, device=DEV), n, k)
    rows = torch.cat([torch.arange(4), torch.arange(65530, 65542), torch.arange(n - 60, n)]).to(DEV)
    few = w4.MXFP4Rows(codes[rows].contiguous(), w.scales[rows].contiguous(), len(rows), k)
    for m in (2, 10, 40, 130):
        a = w4.MXFP4Rows(codes[100:100 + m].contiguous(), w.scales[:m], m, k)
        assert torch.equal(w4.mm_mxfp4(a, w)[:, rows], w4.mm_mxfp4(a, few))
    values = w4.dequantize_mxfp4(w, torch.bfloat16)
    assert torch.equal(values[rows], w4.dequantize_mxfp4(few, torch.bfloat16))
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        dy = torch.zeros(len(rows), n, dtype=dtype, device=DEV)
        dy[torch.arange(len(rows), device=DEV), rows] = 2.0
        assert torch.equal(w4.mm_mxfp4_t(dy, w, out_dtype=torch.bfloat16), 2 * values[rows])
    again = w4.quantize_mxfp4(values)
    assert torch.equal(w4.dequantize_mxfp4(again), values)


GRADS = [(1, 64, 64, 0), (3, 100, 70, 0), (16, 2027, 130, 0), (33, 512, 1030, 8), (64, 8, 2048, 0), (100, 1000, 257, 3),
         (131, 515, 128, 0), (300, 264, 520, 0), (257, 1024, 1024, 0), (520, 320, 4160, 16), (1, 1, 1, 0), (700, 200, 23000, 0),
         (33, 4104, 2080, 0), (1, 8192, 64, 0), (65, 8, 257, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,pad", GRADS)
@pytest.mark.parametrize("dtype", FLOATS)
def test_gradient_formula(m, n, k, pad, dtype):
    dy, dy64 = _rows(m + n, m, n, dtype, pad, scale=0.1)
    w, w64 = _weight(k, n, k)
    ref, size = dy64 @ w64, np.abs(dy64) @ np.abs(w64)
    parts = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}[dtype]
    for out in {dtype, torch.float32}:
        # exact products of each part; their sums in any order, each rounded or cut (2 EPS32)
        _check_rounded(w4.mm_mxfp4_t(dy, w, out_dtype=out), ref, size, out, f"{m}x{n}x{k}", steps=2 * parts * n + 4)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,pad", GRADS)
@pytest.mark.parametrize("dtype", FLOATS)
def test_gradient_rows_alone(m, n, k, pad, dtype):
    """Every contraction row by itself: dY of one number a row gives that row of values, exactly; the
    number has as many bits as its type, so all of its parts count."""
    w, w64 = _weight(n, n, k, spread=20)
    want = torch.from_numpy(w64).to(DEV)
    one = {torch.bfloat16: 1 + 2.0**-7, torch.float16: 1 + 2.0**-10, torch.float32: 1 + 2.0**-7 + 2.0**-15 + 2.0**-23}[dtype]
    for at in range(0, n, m):
        rows = (torch.arange(m, device=DEV) + min(at, max(0, n - m))) % n
        dy = torch.zeros(m, n + pad, dtype=dtype, device=DEV)[:, :n]
        dy[torch.arange(m, device=DEV), rows] = one
        got = w4.mm_mxfp4_t(dy, w).double()
        # two significant bits of w times 24 of dY: one rounding of the sum of exact parts at most
        assert ((got - one * want[rows]).abs() <= 2 * EPS32 * (one * want[rows]).abs()).all(), at
        if dtype != torch.float32:
            assert torch.equal(got, one * want[rows]), at
        if at > 40 * m:
            break


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
def test_gradient_special_values(dtype):
    """Infinities and NaN of dY stay in their row and are what the formula gives; the type's largest and
    least values keep their bits; a NaN block reaches its 32 columns."""
    n, k = 200, 96
    w, w64 = _weight(6, n, k, spread=0)
    w.codes |= 0x11  # no zero codes: 0 times infinity would be NaN
    w64 = w4.dequantize_mxfp4(w, torch.float32).double().cpu().numpy()
    dy = torch.randn(9, n, device=DEV).to(dtype)
    dy[1] = 0
    dy[2, 5], dy[3, 7], dy[4, 0] = float("nan"), float("inf"), -float("inf")
    dy[5], dy[6] = 0, 0
    dy[5, 3], dy[6, 4] = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    y = w4.mm_mxfp4_t(dy, w).double().cpu().numpy()
    assert not y[1].any() and np.isnan(y[2]).all()
    assert (y[3] == np.inf * np.sign(w64[7])).all() and (y[4] == -np.inf * np.sign(w64[0])).all()
    for r, c in ((5, 3), (6, 4)):
        v = float(dy[r, c])
        assert (np.abs(y[r] - v * w64[c]) <= 2 * EPS32 * np.abs(v * w64[c]) + 2.0**-133).all()
    w.scales[11, 1] = 255
    y = w4.mm_mxfp4_t(dy[7:], w).isnan().cpu().numpy()
    assert y[:, 32:64].all() and not y[:, :32].any() and not y[:, 64:].any()


@pytest.mark.gpu
def test_gradient_misaligned_and_strided():
    w, _ = _weight(11, 200, 96)
    buf = torch.randn(50 * 200 + 8, device=DEV).to(torch.bfloat16)
    dy = buf[1:1 + 50 * 200].view(50, 200)  # two bytes off a 16-byte boundary
    assert torch.equal(w4.mm_mxfp4_t(dy, w), w4.mm_mxfp4_t(dy.clone(), w))
    w, _ = _weight(51, 4096, 96)
    dy = torch.empty(8, 1024, 4096, dtype=torch.bfloat16, device=DEV)
    last = dy[:, -1, :]
    last.copy_(torch.randn(8, 4096, device=DEV))
    assert last.stride(0) == 1 << 22
    assert torch.equal(w4.mm_mxfp4_t(last, w), w4.mm_mxfp4_t(last.contiguous(), w))


@pytest.mark.gpu
def test_gradient_differences():
    """Central differences of the product itself: tokens of whole multiples of one power whose largest
    magnitude is 4 keep it, so a step of half a unit moves the output by exactly that."""
    m, n, k = 5, 24, 64
    g = np.random.default_rng(6)
    x = g.integers(-2, 3, (m, k)) * 0.5
    x[:, ::32] = 4
    w, w64 = _weight(12, n, k)
    dy = torch.from_numpy(g.standard_normal((m, n)).astype(np.float32)).to(DEV)
    dx = w4.mm_mxfp4_t(dy, w).double().cpu().numpy()

    def f(a):
        return (dy.double() * w4.mm_mxfp4(torch.from_numpy(a.astype(np.float32)).to(DEV), w).double()).sum(1).cpu().numpy()

    ybig = np.abs(x) @ np.abs(w64).T + 4 * np.abs(w64).max()
    d = dy.double().abs().cpu().numpy()
    for j in range(k):
        if j % 32 == 0:
            continue
        up, dn = x.copy(), x.copy()
        up[:, j] += 0.5
        dn[:, j] -= 0.5
        # fp32 sums of k terms in the two outputs, of 3 n in the gradient
        tol = (d * ybig).sum(1) * 2 * (2 * k + 4) * EPS32 + (d @ np.abs(w64[:, j])) * (6 * n + 4) * EPS32
        assert (np.abs(f(up) - f(dn) - dx[:, j]) <= tol).all(), j


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
def test_layer_autograd(dtype):
    wt = torch.randn(48, 96, device=DEV) * 0.05
    layer = w4.MXFP4Linear.from_weight(wt, bias=torch.randn(48, device=DEV), out_dtype=dtype)
    assert (layer.in_features, layer.out_features) == (96, 48)
    layer.bias.requires_grad_()
    x = torch.randn(2, 7, 96, device=DEV).to(dtype).requires_grad_()
    y = layer(x)
    assert y.shape == (2, 7, 48) and y.dtype == dtype
    gy = torch.randn_like(y)
    y.backward(gy)
    assert torch.equal(x.grad.view(-1, 96), w4.mm_mxfp4_t(gy.view(-1, 48), layer.w, out_dtype=dtype))
    assert torch.allclose(layer.bias.grad.float(), gy.view(-1, 48).float().sum(0).to(dtype).float())
    q = w4.dequantize_mxfp4(w4.quantize_mxfp4(x.detach().view(-1, 96)), torch.float32).double()
    ref = q @ w4.dequantize_mxfp4(layer.w, torch.float32).double().t() + layer.bias.double()
    assert ((y.view(-1, 48).double() - ref).abs() <= HALF_ULP[dtype] * 2 * ref.abs() + 1e-4).all()
    x0 = torch.empty(0, 96, device=DEV, dtype=dtype, requires_grad=True)
    w4.mxfp4_linear(x0, layer.w).sum().backward()
    assert x0.grad.shape == (0, 96)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 4, 12, 48, 160])
def test_streams_and_graph_replays(m):
    w, _ = _weight(31, 256, 1024)
    x = _rows(m, m, 1024, torch.bfloat16)[0].contiguous()
    dy = _rows(m, m, 256, torch.float16)[0].contiguous()

    def both():
        return w4.mm_mxfp4(x, w), w4.mm_mxfp4_t(dy, w), w4.dequantize_mxfp4(w4.quantize_mxfp4(x))

    want = both()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = both()
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(3):
        x.copy_(_rows(100 + i, m, 1024, torch.bfloat16)[0])
        dy.copy_(_rows(200 + i, m, 256, torch.float16)[0])
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,pad", [(0, 5, 0), (1, 1, 0), (3, 257, 0), (127, 40, 3), (128, 256, 0), (1000, 2049, 5), (20000, 33, 0)])
@pytest.mark.parametrize("dtype", FLOATS)
def test_sum_rows(m, n, pad, dtype):
    x = torch.randn(m, n + pad, device=DEV).to(dtype)[:, :n]
    want = x.double().sum(0)
    most = x.double().abs().sum(0)
    for out in FLOATS:
        got = w4.mxfp4.sum_rows(x, out)
        assert got.shape == (n,) and got.dtype == out
        # m fp32 additions, each off by at most half an ulp of a partial sum, and one rounding
        tol = most * (m * EPS32) + want.abs() * HALF_ULP[out] * 1.01 + TINY[out]
        assert ((got.double() - want).abs() <= tol).all(), out
        assert torch.equal(got, w4.mxfp4.sum_rows(x, out))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(5, 64), (2048, 1024), (4096, 96)])
def test_captured_step(m, n):
    """Forward and backward in one graph, the bias's gradient with it, over several replays."""
    w, _ = _weight(33, n, 256)
    x = _rows(m, m, 256, torch.bfloat16)[0].contiguous().requires_grad_()
    bias = torch.randn(n, device=DEV).requires_grad_()
    gy = torch.randn(m, n, device=DEV)

    def step(x, bias):
        y = w4.mxfp4_linear(x, w, bias)
        return y, *torch.autograd.grad(y, (x, bias), gy)

    def eager():  # leaves of its own
        return step(x.detach().clone().requires_grad_(), bias.detach().clone().requires_grad_())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            eager()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, bias)
    for i in range(5):
        with torch.no_grad():
            x.copy_(_rows(300 + i, m, 256, torch.bfloat16)[0])
            bias.copy_(torch.randn(n, device=DEV))
            gy.copy_(torch.randn(m, n, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in out]
        for a, b in zip(got, eager()):
            assert torch.equal(a, b), i


@pytest.mark.gpu
def test_more_rows_than_a_launch_holds():
    """Rows and channels past one launch's: every row the same as its copy among the first."""
    x = torch.randn(64, 64, device=DEV).bfloat16()
    n = (1 << 26) + 192  # 2^30 chunks of eight columns and some
    few, many = w4.quantize_mxfp4(x), w4.quantize_mxfp4(x.repeat(n // 64, 1))
    assert (many.codes.view(-1, 64, 64) == few.codes).all() and (many.scales.view(-1, 64, 4) == few.scales).all()
    values = w4.dequantize_mxfp4(many)
    assert (values.view(-1, 64, 64) == w4.dequantize_mxfp4(few)).all()
    del values
    for a in (x[:3], w4.MXFP4Rows(few.codes[:3], few.scales[:3], 3, 64)):
        y = w4.mm_mxfp4(a, many, out_dtype=torch.bfloat16).view(3, -1, 64)
        assert torch.equal(y[:, 0], w4.mm_mxfp4(a, few, out_dtype=torch.bfloat16)) and (y == y[:, :1]).all()
