"""The 8-bit integer linear operators: refusals on the host, and on the GPU the quantizer
bit for bit, the product against int64 sums, the gradient against its formula in 64 bits
and against differences of the product itself."""

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

    path = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "w8a8.h")
    names = re.findall(r"^(?:int|int64_t|const char\*)\s+(w8\w+|tok\w+)\s*\(", open(path).read(), flags=re.M)
    assert sorted(names) == sorted(_lib.EXPORTS_W8)
    for n in names:
        assert hasattr(w4.lib(), n), n


def test_pitch():
    L = w4.lib()
    assert [L.w8_pitch(k) for k in (0, 1, 64, 65, 11008)] == [-1, 64, 64, 128, 11008]


def test_quantize_refusals():
    q = w4.lib().w8_quantize_rows
    assert q(_p(), 0, 4, 0, 64, _p(), _p(), None) == _lib.W4_ERR_INVALID
    assert q(_p(), 7, 4, 64, 64, _p(), _p(), None) == _lib.W4_ERR_INVALID
    assert q(_p(), 2, -1, 64, 64, _p(), _p(), None) == _lib.W4_ERR_INVALID
    assert q(_p(), 2, 4, 64, 63, _p(), _p(), None) == _lib.W4_ERR_INVALID
    assert q(None, 2, 4, 64, 64, _p(), _p(), None) == _lib.W4_ERR_INVALID
    assert q(_p(), 2, 4, 64, 64, None, _p(), None) == _lib.W4_ERR_INVALID
    assert q(_p(), 2, 4, 1 << 17, 1 << 17, _p(), _p(), None) == _lib.W4_ERR_UNSUPPORTED
    assert q(_p(0x10001), 2, 4, 64, 64, _p(), _p(), None) == _lib.W4_ERR_ALIGN
    assert q(_p(), 2, 4, 64, 64, _p(0x10008), _p(), None) == _lib.W4_ERR_ALIGN
    assert q(None, 2, 0, 64, 64, None, None, None) == _lib.W4_OK


def test_product_refusals():
    def mm(A=_p(), sa=_p(), M=4, W=_p(), sw=_p(), N=64, K=128, bias=None, dt=0, segs=_seg(64), n=1, ws=None, wsb=0):
        return w4.lib().w8a8_mm(A, sa, M, W, sw, N, K, bias, dt, segs, n, ws, wsb, None)

    assert mm(M=-1) == _lib.W4_ERR_INVALID
    assert mm(N=0) == _lib.W4_ERR_INVALID
    assert mm(K=0) == _lib.W4_ERR_INVALID
    assert mm(K=1 << 17) == _lib.W4_ERR_UNSUPPORTED
    assert mm(A=None) == _lib.W4_ERR_INVALID
    assert mm(sw=None) == _lib.W4_ERR_INVALID
    assert mm(W=_p(0x10004)) == _lib.W4_ERR_ALIGN
    assert mm(dt=3) == _lib.W4_ERR_INVALID
    assert mm(segs=_seg(63)) == _lib.W4_ERR_INVALID
    assert mm(segs=_seg(64, ld=60)) == _lib.W4_ERR_INVALID
    assert mm(segs=_seg(64, y=None)) == _lib.W4_ERR_INVALID
    assert mm(n=5) == _lib.W4_ERR_INVALID
    assert mm(bias=_p(0x10002)) == _lib.W4_ERR_ALIGN
    assert mm(ws=_p(0x10004), wsb=64) == _lib.W4_ERR_ALIGN
    assert mm(M=0, A=None) == _lib.W4_OK
    assert "4" in _lib.status_string(_lib.W4_ERR_ALIGN)


def test_linear_and_gradient_refusals():
    L = w4.lib()

    def linear(X=_p(), dt=2, ld=128, M=64, ws=None, wsb=0):
        return L.w8a8_linear(X, dt, ld, M, _p(), _p(), 64, 128, None, 0, _seg(64), 1, ws, wsb, None)

    assert linear(dt=5) == _lib.W4_ERR_INVALID
    assert linear(ld=100) == _lib.W4_ERR_INVALID
    assert linear(X=None) == _lib.W4_ERR_INVALID
    size = ctypes.c_size_t(0)
    assert L.w8a8_workspace_bytes(64, 64, 128, 2, ctypes.byref(size)) == 0 and size.value >= 64 * 128 + 64 * 4
    assert linear() == _lib.W4_ERR_RESOURCE
    assert linear(ws=_p(), wsb=size.value - 1) == _lib.W4_ERR_RESOURCE

    def mt(dY=_p(), dt=2, ld=64, M=4, N=64, K=128, segs=_seg(128), ws=None, wsb=0):
        return L.w8a16_mm_t(dY, dt, ld, M, _p(), _p(), N, K, 0, segs, 1, ws, wsb, None)

    assert mt(dt=0) == _lib.W4_ERR_INVALID
    assert mt(dY=None) == _lib.W4_ERR_INVALID
    assert mt(segs=_seg(64)) == _lib.W4_ERR_INVALID
    assert mt(N=1 << 22, ld=1 << 22) == _lib.W4_ERR_UNSUPPORTED
    assert mt(N=63) == _lib.W4_ERR_RESOURCE  # an unaligned dY needs its copy
    assert mt(dY=_p(0x10002)) == _lib.W4_ERR_RESOURCE
    assert L.w8a16_mm_t_workspace_bytes(4, 63, 128, 63, ctypes.byref(size)) == 0 and size.value >= 4 * 64 * 2


def test_binding_refusals():
    w = w4.Int8Rows(torch.zeros(8, 64, dtype=torch.int8), torch.ones(8), 8, 64)
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="HIP device"):
        w4.mm_int8(x, w)
    with pytest.raises(ValueError, match="width"):
        w4.mm_int8(torch.zeros(2, 63), w)
    with pytest.raises(TypeError):
        w4.mm_int8(torch.zeros(2, 64, dtype=torch.float64), w)
    with pytest.raises(ValueError, match="bias"):
        w4.mm_int8(x, w, bias=torch.zeros(7))
    with pytest.raises(ValueError, match="out must"):
        w4.mm_int8(x, w, out=torch.zeros(2, 9))
    with pytest.raises(ValueError, match="codes"):
        w4.mm_int8(x, w4.Int8Rows(torch.zeros(8, 63, dtype=torch.int8), torch.ones(8), 8, 63))
    with pytest.raises(ValueError, match="scales"):
        w4.mm_int8(x, w4.Int8Rows(torch.zeros(8, 64, dtype=torch.int8), torch.ones(7), 8, 64))
    with pytest.raises(ValueError, match="sum to"):
        w4.mm_int8_split(x, w, [torch.zeros(2, 3)])
    with pytest.raises(TypeError):
        w4.mm_int8_t(torch.zeros(2, 8), w)
    with pytest.raises(ValueError, match="width"):
        w4.mm_int8_t(torch.zeros(2, 9, dtype=torch.bfloat16), w)
    with pytest.raises(ValueError, match="out_dtype"):
        w4.W8A8Linear(w, out_dtype=torch.int8)


# ---------------------------------------------------------------- GPU


def _rows(seed, rows, cols, dtype, pad=0, scale=1.0):
    """Seeded rows with per-row magnitudes, as (device tensor of rows `pad` longer, fp32 numpy)."""
    g = np.random.default_rng(seed)
    a = g.standard_normal((rows, cols)) * np.exp(g.standard_normal((rows, 1))) * scale
    t = torch.from_numpy(a.astype(np.float32)).to(dtype)
    wide = torch.full((rows, cols + pad), float("nan"), dtype=dtype)
    wide[:, :cols] = t
    return wide.to(DEV)[:, :cols], t.float().numpy()


def _quantize_ref(x32):
    """The definition in IEEE fp32, step by step."""
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.abs(x32).max(axis=1)
        s = np.maximum(a / np.float32(127), np.float32(2.0**-126)).astype(np.float32)
        q = np.rint(x32 * (np.float32(1) / s)[:, None])
    bad = ~np.isfinite(x32).all(axis=1)
    s[bad] = np.nan
    q[bad] = 0
    return q.astype(np.int8), s


def _weight(seed, n, k):
    g = np.random.default_rng(seed)
    codes = np.zeros((n, (k + 63) // 64 * 64), dtype=np.int8)
    codes[:, :k] = g.integers(-127, 128, (n, k), dtype=np.int8)
    scales = (0.001 * np.exp(0.5 * g.standard_normal(n))).astype(np.float32)
    w = w4.Int8Rows(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), n, k)
    return w, codes[:, :k].astype(np.int64), scales.astype(np.float64)


def _check_rounded(y, ref, size, dtype, what, steps=4):
    """|y - ref| <= `steps` fp32 roundings of magnitude `size`, and one rounding to dtype."""
    y = y.double().cpu().numpy()
    tol = steps * EPS32 * size + (HALF_ULP[dtype] * (np.abs(ref) + steps * EPS32 * size) + TINY[dtype]
                                  if dtype != torch.float32 else 0.0)
    bad = ~(np.abs(y - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {np.abs(y - ref)[bad].max():.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 7, 1), (5, 64, 0), (2, 65, 3), (9, 2048, 0), (4, 2049, 5),
                                           (3, 8191, 0), (7, 11008, 0), (2, 16385, 0), (1, 70001, 2)])
def test_quantize_bits(dtype, rows, cols, pad):
    x, x32 = _rows(rows * 1000 + cols, rows, cols, dtype, pad)
    r = w4.quantize_int8(x)
    q, s = _quantize_ref(x32)
    np.testing.assert_array_equal(r.scales.cpu().numpy(), s)
    got = r.codes.cpu().numpy()
    np.testing.assert_array_equal(got[:, :cols], q)
    assert not got[:, cols:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_quantize_special_rows(dtype):
    x32 = np.random.default_rng(3).standard_normal((7, 100)).astype(np.float32)
    x32[0] = 0
    x32[1, 17] = np.nan
    x32[2, 99] = np.inf
    x32[3, 0] = -np.inf
    x32[4] = 2.0**-130 if dtype != torch.float16 else 2.0**-24  # below the least normal fp32 (or fp16)
    x32[5, :] = 1.0
    x32[6, 5] = torch.finfo(dtype).max
    t = torch.from_numpy(x32).to(dtype)
    r = w4.quantize_int8(t.to(DEV))
    q, s = _quantize_ref(t.float().numpy())
    np.testing.assert_array_equal(r.scales.cpu().numpy(), s)
    np.testing.assert_array_equal(r.codes.cpu().numpy()[:, :100], q)
    w, _, _ = _weight(1, 16, 100)
    y = w4.mm_int8(t.to(DEV), w).cpu().numpy()
    assert np.isnan(y[1:4]).all() and np.isfinite(y[[0, 4, 5, 6]]).all() and not y[0].any()


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 2048, 2048), (2, 33, 70), (3, 1000, 4096), (4, 512, 11008), (5, 100, 129),
          (16, 48, 4096), (17, 515, 2048), (32, 256, 1030), (33, 130, 640), (64, 96, 8192), (65, 300, 1000),
          (127, 257, 511), (128, 128, 128), (200, 640, 192), (257, 259, 300), (300, 1003, 1555), (515, 2050, 257)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_product(m, n, k, dtype):
    """Float activations and int8 rows give the same bits, equal to the int64 sums scaled."""
    x, x32 = _rows(m + n + k, m, k, dtype, pad=3 if m % 2 else 0)
    w, codes, scales = _weight(n + k, n, k)
    bias = torch.from_numpy(np.random.default_rng(5).standard_normal(n).astype(np.float32)).to(dtype)
    y = w4.mm_int8(x, w, bias=bias.to(DEV), out_dtype=dtype)
    xq = w4.quantize_int8(x)
    y2 = w4.mm_int8(xq, w, bias=bias.to(DEV), out_dtype=dtype)
    assert torch.equal(y, y2)
    q, s = _quantize_ref(x32)
    prod = (q.astype(np.int64) @ codes.T).astype(np.float64) * s.astype(np.float64)[:, None] * scales
    b = bias.double().numpy()
    # conversion of the sum, two products, the bias
    _check_rounded(y, prod + b, np.abs(prod) + np.abs(b), dtype, f"{m}x{n}x{k}")
    y3 = w4.mm_int8(xq, w)
    _check_rounded(y3, prod, np.abs(prod), torch.float32, f"{m}x{n}x{k} fp32")
    assert torch.equal(w4.mm_int8(xq, w), y3)  # the same bits again


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(700, 23000, 640), (3000, 8192, 2048), (1500, 8600, 1030), (2048, 11008, 4096),
                                   (2060, 9000, 520)])
def test_product_mixed_tiles(m, n, k):
    """Whole rounds of 256-row tiles and lower ones for the columns left, where the plan says so."""
    g = torch.Generator(device=DEV).manual_seed(m + n)
    a, w = (w4.quantize_int8(torch.randn(r, k, device=DEV, generator=g)) for r in (m, n))
    y = w4.mm_int8(a, w)
    # exact in double
    ref = (a.codes.double() @ w.codes.double().t()) * a.scales.double()[:, None] * w.scales.double()
    assert ((y.double() - ref).abs() <= ref.abs() * 2.0**-22).all()  # three fp32 roundings
    assert torch.equal(w4.mm_int8(a, w), y)


def test_split_without_outputs():
    w = w4.Int8Rows(torch.zeros(8, 64, dtype=torch.int8), torch.ones(8), 8, 64)
    with pytest.raises(ValueError, match="at least one output"):
        w4.mm_int8_split(torch.zeros(2, 64), w, [])


def test_product_plans():
    names = [w4.int8_kernel_for(*s) for s in ((3000, 8192, 2048), (2048, 11008, 4096), (8192, 8192, 8192))]
    assert "+" in names[0] and "+" in names[1] and names[2] == "w8_256x256"


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 2, 20, 130])
def test_product_extreme_codes(m):
    """Sums near the int32 limit: K = 131071 codes of -128 and 127."""
    k, n = 131071, 5
    codes = torch.full((n, 131072), -128, dtype=torch.int8)
    codes[:, k:] = 0
    codes[1] = -codes[1].to(torch.int16).clamp(-127, 127).to(torch.int8)
    a = torch.full((m, 131072), -128, dtype=torch.int8)
    a[:, k:] = 0
    w = w4.Int8Rows(codes.to(DEV), torch.ones(n, device=DEV), n, k)
    y = w4.mm_int8(w4.Int8Rows(a.to(DEV), torch.ones(m, device=DEV), m, k), w).cpu()
    ref = (a[0].long() * codes.long()).sum(1).float()
    assert torch.equal(y, ref.expand(m, n))


@pytest.mark.gpu
def test_product_split_outputs_and_views():
    m, k = 37, 320
    w, _, _ = _weight(8, 24 + 8 + 9, k)
    x, _ = _rows(4, m, k, torch.bfloat16)
    whole = w4.mm_int8(x, w, out_dtype=torch.bfloat16)
    bufs = [torch.full((m, c + 5), 7.0, dtype=torch.bfloat16, device=DEV) for c in (24, 8, 9)]
    w4.mm_int8_split(x, w, [b[:, 2:-3] for b in bufs])
    assert torch.equal(torch.cat([b[:, 2:-3] for b in bufs], 1), whole)
    for b in bufs:
        assert (b[:, :2] == 7).all() and (b[:, -3:] == 7).all()
    for mm in (1, 4, 40):  # rows before and after the output stay as they are
        x, _ = _rows(mm, mm, k, torch.bfloat16)
        guard = torch.full((mm + 2, 41), 3.0, device=DEV)
        w4.mm_int8(x, w, out=guard[1:-1])
        assert (guard[0] == 3).all() and (guard[-1] == 3).all() and (guard[1:-1] != 3).any()


@pytest.mark.gpu
def test_product_no_rows():
    w, _, _ = _weight(2, 8, 64)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    assert w4.mm_int8(x, w).shape == (0, 8)
    assert w4.mm_int8_t(torch.empty(0, 8, dtype=torch.bfloat16, device=DEV), w).shape == (0, 64)
    assert w4.quantize_int8(x).codes.shape == (0, 64)


@pytest.mark.gpu
def test_product_far_offsets():
    """A weight of more than 2^31 bytes."""
    n, k = 70003, 32768
    codes = torch.randint(-127, 128, (n, k), dtype=torch.int8, device=DEV)
    scales = torch.rand(n, device=DEV) + 0.5
    w = w4.Int8Rows(codes, scales, n, k)
    for m in (2, 40, 130):
        x = torch.randn(m, k, device=DEV)
        xq = w4.quantize_int8(x)
        y = w4.mm_int8(xq, w)
        rows = torch.cat([torch.arange(4), torch.arange(65530, 65540), torch.arange(n - 60, n)]).to(DEV)
        ref = (xq.codes.double() @ codes[rows].double().t()) * xq.scales.double()[:, None] * scales[rows].double()
        _check_rounded(y[:, rows], ref.cpu().numpy(), ref.abs().cpu().numpy(), torch.float32, f"m={m}")


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,pad", [(1, 64, 64, 0), (3, 100, 70, 0), (16, 2027, 130, 0), (33, 512, 1030, 8),
                                       (64, 8, 2048, 0), (100, 1000, 257, 3), (131, 515, 128, 0), (300, 264, 520, 0),
                                       (257, 1024, 1024, 0), (520, 320, 4160, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradient_formula(m, n, k, pad, dtype):
    dy, dy32 = _rows(m + n, m, n, dtype, pad, scale=0.1)
    w, codes, _ = _weight(k, n, k)
    s32 = w.scales.cpu().numpy()
    op = torch.from_numpy(codes.astype(np.float32) * s32[:, None]).to(dtype).double().numpy()
    ref = dy32.astype(np.float64) @ op
    size = np.abs(dy32).astype(np.float64) @ np.abs(op)
    for out in (dtype, torch.float32):
        # n products and as many additions in fp32, in any order
        _check_rounded(w4.mm_int8_t(dy, w, out_dtype=out), ref, size, out, f"{m}x{n}x{k}", steps=n + 2)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,pad,dtype", [
    (700, 200, 23000, 0, torch.bfloat16),   # whole rounds of tall tiles, the columns left in lower ones
    (513, 72, 33000, 8, torch.float16), (2048, 136, 11008, 0, torch.float16),
    (300, 1000, 5000, 0, torch.bfloat16), (33, 4104, 2080, 0, torch.float16),  # split contractions
    (130, 2027, 515, 3, torch.bfloat16), (1, 8192, 64, 0, torch.bfloat16), (65, 8, 257, 0, torch.float16)])
def test_gradient_plans(m, n, k, pad, dtype):
    test_gradient_formula(m, n, k, pad, dtype)


@pytest.mark.gpu
def test_gradient_misaligned():
    w, _, _ = _weight(11, 200, 96)
    buf = torch.randn(50 * 200 + 8, device=DEV).to(torch.bfloat16)
    dy = buf[1:1 + 50 * 200].view(50, 200)  # two bytes off a 16-byte boundary
    assert torch.equal(w4.mm_int8_t(dy, w), w4.mm_int8_t(dy.clone(), w))


@pytest.mark.gpu
def test_gradient_differences():
    """Central differences of the product itself: integer tokens with a 127 in each row have scale
    1, so a step of one in another entry moves the output by exactly one code's worth."""
    m, n, k = 5, 24, 40
    g = np.random.default_rng(6)
    x = g.integers(-60, 61, (m, k)).astype(np.float32)
    x[:, 0] = 127
    w, _, _ = _weight(12, n, k)
    dy = torch.from_numpy(g.standard_normal((m, n)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    dx = w4.mm_int8_t(dy, w).double().cpu().numpy()

    def f(a):
        return (dy.double() * w4.mm_int8(torch.from_numpy(a).to(DEV), w).double()).sum(1).cpu().numpy()

    wop = np.abs(w.codes.cpu().numpy()[:, :k] * w.scales.cpu().numpy()[:, None].astype(np.float64))
    ybig = np.abs(x).astype(np.float64) @ wop.T
    dyn = dy.double().abs().cpu().numpy()
    for j in range(1, k):
        up, dn = x.copy(), x.copy()
        up[:, j] += 1
        dn[:, j] -= 1
        # the weight operand's rounding to bf16, and the fp32 rounding of the two outputs
        tol = (dyn @ wop[:, j]) * (2.0**-8 + 30 * EPS32) + (dyn * (ybig + 127 * wop.max())).sum(1) * 4 * EPS32
        assert (np.abs((f(up) - f(dn)) / 2 - dx[:, j]) <= tol).all(), j


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_layer_autograd(dtype):
    wt = torch.randn(48, 96, device=DEV) * 0.05
    layer = w4.W8A8Linear.from_weight(wt, bias=torch.randn(48, device=DEV), out_dtype=dtype)
    layer.bias.requires_grad_()
    x = torch.randn(2, 7, 96, device=DEV).to(dtype).requires_grad_()
    y = layer(x)
    assert y.shape == (2, 7, 48) and y.dtype == dtype
    gy = torch.randn_like(y)
    y.backward(gy)
    g16 = gy if dtype != torch.float32 else gy.to(torch.bfloat16)
    assert torch.equal(x.grad.view(-1, 96), w4.mm_int8_t(g16.view(-1, 48), layer.w, out_dtype=dtype))
    assert torch.allclose(layer.bias.grad.float(), gy.view(-1, 48).float().sum(0).to(dtype).float())
    # the int8 product is within one half code a term of the float one
    ref = torch.nn.functional.linear(x.double(), wt.double(), layer.bias.double())
    assert ((y.double() - ref).norm() / ref.norm()).item() < 0.03


@pytest.mark.gpu
def test_other_stream():
    w, _, _ = _weight(21, 128, 512)
    st = torch.cuda.Stream()
    for m in (2, 70):
        x, _ = _rows(m, m, 512, torch.bfloat16)
        want = w4.mm_int8(x, w)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            got = w4.mm_int8(x, w)
        st.synchronize()
        assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 48, 160])
def test_graph_replays(m):
    w, _, _ = _weight(31, 256, 1024)
    x, _ = _rows(m, m, 1024, torch.bfloat16)
    x = x.contiguous()
    w4.mm_int8(x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = w4.mm_int8(x, w)
    for i in range(3):
        x.copy_(_rows(100 + i, m, 1024, torch.bfloat16)[0])
        want = w4.mm_int8(x, w)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.gpu
def test_more_rows_than_a_launch_holds():
    """Rows and channels past one launch's: every row the same as its copy among the first."""
    x = torch.randn(64, 64, device="cuda").bfloat16()
    n = (1 << 21) + 192
    few, many = w4.quantize_int8(x), w4.quantize_int8(x.repeat(n // 64, 1))
    assert (many.codes.view(-1, 64, 64) == few.codes).all() and (many.scales.view(-1, 64) == few.scales).all()
    n = (1 << 25) + 64
    w = w4.Int8Rows(few.codes.repeat(n // 64, 1), few.scales.repeat(n // 64), n, 64)
    for a in (x[:3], w4.Int8Rows(few.codes[:3], few.scales[:3], 3, 64)):
        y = w4.mm_int8(a, w, out_dtype=torch.bfloat16).view(3, -1, 64)
        assert torch.equal(y[:, 0], w4.mm_int8(a, few, out_dtype=torch.bfloat16)) and (y == y[:, :1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(5, 40, 70), (131, 515, 128), (33, 4104, 2080), (513, 72, 33000)])
@pytest.mark.parametrize("power", [-100, -40, -24, 12, 24, 100])
def test_gradient_of_any_scale(m, n, k, power):
    """A power of two in all of the weight's scales is one in the result, bit for bit: fp16 gradients
    of weights whose values fp16 does not hold."""
    dy, _ = _rows(m + n, m, n, torch.float16, scale=0.1)
    w, _, _ = _weight(k, n, k)
    other = w4.Int8Rows(w.codes, w.scales * 2.0**power, n, k)
    want = w4.mm_int8_t(dy, w).double() * 2.0**power
    assert torch.equal(w4.mm_int8_t(dy, other).double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(7, 200, 96), (64, 1000, 257), (300, 4104, 520)])
def test_gradient_of_mixed_scales(m, n, k):
    """Channels whose scales are up to 2^20 apart: every operand keeps fp16's eleven bits."""
    dy, dy32 = _rows(m * n, m, n, torch.float16, scale=0.1)
    w, codes, s = _weight(n, n, k)
    w.scales *= torch.from_numpy(2.0 ** -np.random.default_rng(n).integers(0, 20, n).astype(np.float32)).to(DEV) * 2.0**-6
    w.scales[3] = 0.0
    s = w.scales.double().cpu().numpy()
    ref = dy32.astype(np.float64) @ (codes * s[:, None])
    size = np.abs(dy32).astype(np.float64) @ np.abs(codes * s[:, None])
    # the operand's rounding (2^-11), n products and as many additions in fp32
    _check_rounded(w4.mm_int8_t(dy, w), ref, size, torch.float32, f"{m}x{n}x{k}", steps=2.0**13 + n + 2)
    # the small channels alone: the large ones' gradients are 0
    small = torch.from_numpy(s < s.max() * 2.0**-12).to(DEV)
    alone = torch.where(small, dy, torch.zeros_like(dy))
    a64 = alone.double().cpu().numpy()
    ref, size = a64 @ (codes * s[:, None]), np.abs(a64) @ np.abs(codes * s[:, None])
    _check_rounded(w4.mm_int8_t(alone, w), ref, size, torch.float32, f"small {m}x{n}x{k}", steps=2.0**13 + n + 2)


@pytest.mark.gpu
def test_gradient_of_bad_scales():
    """A NaN among a weight's scales makes every result NaN, whatever the other channels hold."""
    for dtype in (torch.float16, torch.bfloat16):
        w, _, _ = _weight(4, 100, 70)
        dy, _ = _rows(1, 9, 100, dtype)
        w.scales[7] = float("nan")
        assert torch.isnan(w4.mm_int8_t(dy, w)).all()
        w.scales[:] = 0.0
        assert not w4.mm_int8_t(dy, w).any()


@pytest.mark.gpu
@pytest.mark.parametrize("x_dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
def test_layer_gradient_keeps_its_type(x_dtype, out_dtype):
    """A 16-bit gradient is multiplied as it is, whatever the activations' type."""
    w, _, _ = _weight(41, 72, 130)
    x = torch.randn(9, 130, device=DEV).to(x_dtype).requires_grad_()
    gy = (torch.randn(9, 72, device=DEV) * 0.1).to(out_dtype)
    w4.w8a8_linear(x, w, out_dtype=out_dtype).backward(gy)
    assert torch.equal(x.grad, w4.mm_int8_t(gy, w, out_dtype=x_dtype))


@pytest.mark.gpu
def test_layer_gradient_range():
    """fp16 activations with an fp32 output: rows of its gradient far below and above fp16's range."""
    m, n, k = 24, 515, 130
    w, codes, _ = _weight(43, n, k)
    x = torch.randn(m, k, device=DEV).half().requires_grad_()
    power = np.linspace(-33, 33, m).round()
    gy = np.random.default_rng(2).standard_normal((m, n)) * 2.0 ** power[:, None]
    gy[5], gy[6, 1:] = 0, 0
    gy = torch.from_numpy(gy.astype(np.float32))
    op = codes * w.scales.double().cpu().numpy()[:, None]
    for row in range(m):  # a weight that brings the row's result back into fp16's range
        wr = w4.Int8Rows(w.codes, w.scales * 2.0 ** -power[row], n, k)
        x.grad = None
        w4.w8a8_linear(x[row:row + 1], wr).backward(gy[row:row + 1].to(DEV))
        r64, o64 = gy[row:row + 1].double().numpy(), op * 2.0 ** -power[row]
        ref, size = r64 @ o64, np.abs(r64) @ np.abs(o64)
        # dY's and the weight's rounding (2^-11 each) and 2^-39 of the row's largest dY, n products and sums in fp32
        floor = np.abs(r64).max() * np.abs(o64).sum(0) * 2.0**-39
        _check_rounded(x.grad[row:row + 1], ref, size + floor * 2.0**11, torch.float16, f"row {row}", steps=2.0**14 + n + 2)
    x.grad = None
    gy[3, 7], gy[4, 8] = float("nan"), float("inf")
    w4.w8a8_linear(x, w).backward(gy.to(DEV))
    bad = ~torch.isfinite(gy).all(1)
    assert not torch.isfinite(x.grad[bad]).any() and not x.grad[5].any()
    x0 = torch.empty(0, k, device=DEV, dtype=torch.float16, requires_grad=True)
    w4.w8a8_linear(x0, w).backward(torch.empty(0, n, device=DEV))
    assert x0.grad.shape == (0, k)


def test_second_derivatives_raise(monkeypatch):
    """The layer's gradient is no function that autograd knows: a second derivative through it raises.
    (The launches are replaced by torch on the CPU: what is left is the autograd.)"""
    from gemv_int4_quantize_amd import int8

    def value(w):
        return w.codes[:, :w.cols].float() * w.scales[:, None]

    monkeypatch.setattr(int8, "mm_int8", lambda x, w, bias=None, out_dtype=None: x.float() @ value(w).t())
    monkeypatch.setattr(int8, "mm_int8_t", lambda g, w, out_dtype=torch.float32: (g.float() @ value(w)).to(out_dtype))
    monkeypatch.setattr(int8, "gradient_of_fp32", lambda g, w, out_dtype: (g @ value(w)).to(out_dtype))
    w = w4.Int8Rows(torch.ones(8, 64, dtype=torch.int8), torch.ones(8), 8, 64)
    bias = torch.zeros(8, requires_grad=True)
    for b in (None, bias):
        x = torch.randn(3, 64, requires_grad=True)
        y = w4.w8a8_linear(x, w, b)
        loss = y.square().sum() + (x**3).sum()
        (g,) = torch.autograd.grad(loss, x, create_graph=True)
        with pytest.raises(RuntimeError, match="twice|once_differentiable"):
            g.square().sum().backward()
        # of a constant dY the result is constant in x: no term is missing
        x = torch.randn(3, 64, requires_grad=True)
        (g,) = torch.autograd.grad(w4.w8a8_linear(x, w, b).sum() + (x**3).sum(), x, create_graph=True)
        assert torch.allclose(torch.autograd.grad(g.sum(), x)[0], 6 * x)
    for dtype in (torch.float16, torch.bfloat16):  # the first derivative, with its graph
        x = torch.randn(3, 64).to(dtype).requires_grad_()
        (g,) = torch.autograd.grad(w4.w8a8_linear(x, w).square().sum(), x, create_graph=True)
        assert g.dtype == dtype and g.requires_grad
    x = torch.randn(3, 64, requires_grad=True)
    w4.w8a8_linear(x, w, bias).sum().backward()
    assert (x.grad == 8).all() and (bias.grad == 3).all()


def test_gradient_workspace_of_long_strides():
    """The reported workspace is what the call asks for, at every row stride."""
    L = w4.lib()
    for M, N, ld in ((4, 64, 1 << 22), (4, 64, (1 << 22) - 8), (4, 64, (1 << 40)), (4, 64, 68), (4, 60, 60), (4, 64, -1),
                     (1, 64, 1 << 22), (1, 64, 67), (1, 60, 64), (2, 64, (1 << 22) - 4)):
        size = ctypes.c_size_t(0)
        assert L.w8a16_mm_t_workspace_bytes(M, N, 128, ld, ctypes.byref(size)) == 0
        copied = N % 8 != 0 or (ld % 8 != 0 or ld >= 1 << 22 if M > 1 else False) or ld < 0
        assert (size.value >= M * 64 * 2) == copied, (M, N, ld)
        if copied and ld > 0:
            status = L.w8a16_mm_t(_p(), 2, ld, M, _p(), _p(), N, 128, 0, _seg(128), 1, _p(), M * 64 * 2 - 1, None)
            assert status == _lib.W4_ERR_RESOURCE, (M, N, ld)
            assert "workspace" in L.w4_last_error().decode()


@pytest.mark.gpu
def test_gradient_long_strides():
    """The last tokens of long sequences: rows 2^22 elements apart."""
    w, _, _ = _weight(51, 4096, 96)
    dy = torch.empty(8, 1024, 4096, dtype=torch.bfloat16, device=DEV)
    last = dy[:, -1, :]
    last.copy_(torch.randn(8, 4096, device=DEV))
    assert last.stride(0) == 1 << 22
    assert torch.equal(w4.mm_int8_t(last, w), w4.mm_int8_t(last.contiguous(), w))
    assert torch.equal(w4.mm_int8_t(last[:1], w), w4.mm_int8_t(last[:1].contiguous(), w))


def test_kernel_names():
    """The name is that of the kernel launched: int8 rows never take the form that quantizes."""
    k = w4.lib().w8a8_kernel
    assert k(2, 4096, 4096, -1) == b"w8_decode" and k(2, 4096, 4096, _lib.DT_BF16) == b"w8_decode_fused"
    assert k(4, 4096, 70000, _lib.DT_BF16) == b"w8_decode"  # codes that LDS does not hold: quantized before
    assert k(64, 4096, 4096, -1) == k(64, 4096, 4096, _lib.DT_F32) is not None
    for bad in ((2, 4096, 4096, 9), (0, 64, 64, -1), (4, 0, 64, -1), (4, 64, 1 << 17, -1)):
        assert k(*bad) is None
    assert w4.int8_kernel_for(1, 2048, 2048) == "w8_decode_fused"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 31, 33, 63, 64, 65, 129, 192, 193, 320])
def test_decode_short_rows(k, dtype):
    """Few columns: codes of half a unit, and the last unit of a pitch that is not a multiple of 128."""
    for m in (1, 2, 3, 4):
        for n in (1, 16, 37, 9000):
            test_product(m, n, k, dtype)


EXACT = [(33, 4104, 2080), (1, 200, 70), (16, 2027, 130), (300, 1000, 520), (600, 515, 23000), (64, 8200, 257)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", EXACT)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradient_rows_alone(m, n, k, dtype):
    """Every contraction row by itself: dY of one 1 a row gives that row of codes, exactly, wherever
    it lies in a stage or a slice of the contraction."""
    w, codes, _ = _weight(n, n, k)
    w.scales[:] = 1.0
    want = torch.from_numpy(codes).to(DEV).float()
    for at in range(0, n, m):
        rows = torch.arange(m, device=DEV) + min(at, max(0, n - m))
        rows %= n
        dy = torch.zeros(m, n, dtype=dtype, device=DEV)
        dy[torch.arange(m, device=DEV), rows] = 1.0
        assert torch.equal(w4.mm_int8_t(dy, w), want[rows]), at


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", EXACT)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradient_whole_numbers(m, n, k, dtype):
    """Small whole numbers: every partial sum is exact in fp32, in any order."""
    w, codes, _ = _weight(n + 1, n, k)
    w.scales[:] = 1.0
    dy = torch.from_numpy(np.random.default_rng(m).integers(-3, 4, (m, n)).astype(np.float32))
    assert 3 * 127 * n < 1 << 24
    ref = dy.double().to(DEV) @ torch.from_numpy(codes).double().to(DEV)
    assert torch.equal(w4.mm_int8_t(dy.to(dtype).to(DEV), w).double(), ref)


@pytest.mark.gpu
def test_gradient_far_offsets():
    """A weight of more than 2^31 bytes: rows of its codes alone, from either side of 2^31."""
    n, k = 70003, 32768
    codes = torch.randint(-127, 128, (n, k), dtype=torch.int8, device=DEV)
    w = w4.Int8Rows(codes, torch.ones(n, device=DEV), n, k)
    rows = torch.cat([torch.arange(4), torch.arange(65530, 65542), torch.arange(n - 24, n)]).to(DEV)
    for dtype in (torch.bfloat16, torch.float16):
        dy = torch.zeros(len(rows), n, dtype=dtype, device=DEV)
        dy[torch.arange(len(rows), device=DEV), rows] = 2.0
        assert torch.equal(w4.mm_int8_t(dy, w, out_dtype=dtype), 2 * codes[rows].to(dtype))


@pytest.mark.gpu
def test_gradient_segments():
    """Several outputs side by side, rows of wider buffers, from the C entry."""
    w, _, _ = _weight(61, 200, 96)
    dy, _ = _rows(3, 40, 200, torch.bfloat16)
    dy = dy.contiguous()
    whole = w4.mm_int8_t(dy, w)
    bufs = [torch.full((40, c + 3), 5.0, device=DEV) for c in (32, 7, 57)]
    segs = (_lib.W4OutSeg * 3)(*[(b.data_ptr() + 4, b.shape[1] - 3, b.shape[1]) for b in bufs])
    st = torch.cuda.current_stream().cuda_stream
    size = ctypes.c_size_t(0)
    assert w4.lib().w8a16_mm_t_workspace_bytes(40, 200, 96, 200, ctypes.byref(size)) == 0
    ws = torch.empty(max(16, size.value), dtype=torch.uint8, device=DEV)
    assert w4.lib().w8a16_mm_t(dy.data_ptr(), _lib.DT_BF16, 200, 40, w.codes.data_ptr(), w.scales.data_ptr(), 200, 96,
                               _lib.DT_F32, segs, 3, ws.data_ptr(), size.value, st) == 0
    assert torch.equal(torch.cat([b[:, 1:-2] for b in bufs], 1), whole)
    for b in bufs:
        assert (b[:, 0] == 5).all() and (b[:, -2:] == 5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", [(32, 4096, 512), (131, 1003, 515)])
def test_gradient_stream_and_graph(m, n, k, dtype):
    w, _, _ = _weight(71, n, k)
    dy = _rows(1, m, n, dtype)[0].contiguous()
    want = w4.mm_int8_t(dy, w)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = w4.mm_int8_t(dy, w)
    st.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx = w4.mm_int8_t(dy, w)
    for i in range(3):
        dy.copy_(_rows(200 + i, m, n, dtype)[0])
        want = w4.mm_int8_t(dy, w)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want)


def test_fp32_gradient_refusals():
    def mt(dY=_p(), ld=64, M=4, N=64, K=128, segs=_seg(128), ws=_p(), wsb=1 << 20):
        return w4.lib().w8a32_mm_t(dY, ld, M, _p(), _p(), N, K, 0, segs, 1, ws, wsb, None)

    assert mt(dY=None) == _lib.W4_ERR_INVALID
    assert mt(dY=_p(0x10002)) == _lib.W4_ERR_ALIGN
    assert mt(ld=63) == _lib.W4_ERR_INVALID
    assert mt(segs=_seg(64)) == _lib.W4_ERR_INVALID
    assert mt(N=1 << 22, ld=1 << 22) == _lib.W4_ERR_UNSUPPORTED
    assert mt(ws=_p(0x10008)) == _lib.W4_ERR_ALIGN
    assert mt(M=0, dY=None, ws=None, wsb=0) == _lib.W4_OK
    size = ctypes.c_size_t(0)
    assert w4.lib().w8a32_mm_t_workspace_bytes(4, 63, 128, ctypes.byref(size)) == 0 and size.value >= 4 * 64 * 2 + 4 * 4
    assert mt(wsb=4 * 64 * 2 + 255) == _lib.W4_ERR_RESOURCE and mt(ws=None) == _lib.W4_ERR_RESOURCE


def _fp32_gradient(dy, w):
    """The definition by way of the fp16 gradient: rows at their powers of two, results taken back.
    (The powers on the host: the device's pow and ldexp of them are not exact.)"""
    d = dy.cpu().numpy()
    e = np.minimum(15 - np.frexp(np.abs(d).max(axis=1, keepdims=True))[1], 126)
    half = torch.from_numpy(np.ldexp(d, e).astype(np.float16)).to(DEV)
    y = np.ldexp(w4.mm_int8_t(half, w).double().cpu().numpy(), -e)
    return torch.from_numpy(y).float().to(DEV)  # the result is fp32: so is its range


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,pad", [(1, 1, 1, 0), (1, 64, 64, 0), (3, 100, 70, 3), (33, 4104, 2080, 0), (131, 2027, 515, 1),
                                       (300, 1000, 520, 8), (16, 9001, 130, 0), (513, 72, 33000, 5), (5, 70001, 64, 0)])
def test_fp32_gradient(m, n, k, pad):
    from gemv_int4_quantize_amd.int8 import gradient_of_fp32

    dy, _ = _rows(m + n, m, n, torch.float32, pad, scale=0.1)
    if not pad:
        dy = torch.from_numpy(np.ldexp(dy.cpu().numpy(), np.linspace(-60, 60, m).round().astype(int)[:, None])).to(DEV)
    w, _, _ = _weight(k, n, k)
    ref = _fp32_gradient(dy.contiguous(), w)
    got = gradient_of_fp32(dy, w, torch.float32)
    assert torch.equal(got, ref)
    for dtype in (torch.float16, torch.bfloat16):
        assert torch.equal(gradient_of_fp32(dy, w, dtype), ref.to(dtype))
    far = w4.Int8Rows(w.codes, w.scales * 2.0**-90, n, k)  # neither power alone would do
    up = dy * 2.0**60 if pad else dy.clamp(-1e15, 1e15) * 2.0**60
    assert torch.equal(gradient_of_fp32(up, far, torch.float32), _fp32_gradient(up.contiguous(), far))


@pytest.mark.gpu
def test_fp32_gradient_special_rows_and_replays():
    from gemv_int4_quantize_amd.int8 import gradient_of_fp32

    w, _, _ = _weight(6, 200, 96)
    w.codes[:, :96][w.codes[:, :96] == 0] = 1
    dy = torch.randn(9, 200, device=DEV)
    dy[1] = 0
    dy[2, 5], dy[3, 7], dy[4, 0] = float("nan"), float("inf"), -float("inf")
    dy[5], dy[6], dy[7] = 3e38, 2.0**-126, 2.0**-140
    got = gradient_of_fp32(dy, w, torch.float32)
    assert not got[1].any() and torch.isnan(got[2]).all() and torch.isinf(got[3:5]).all()
    assert (got[3].sign() == w.codes[7, :96].sign()).all() and (got[4].sign() == -w.codes[0, :96].sign()).all()
    assert torch.equal(got[5:7], _fp32_gradient(dy[5:7], w)) and got[7].abs().max() < 2.0**-126
    assert gradient_of_fp32(dy[:0], w, torch.float32).shape == (0, 96)
    graph = torch.cuda.CUDAGraph()
    x = torch.randn(40, 200, device=DEV)
    gradient_of_fp32(x, w, torch.float16)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = gradient_of_fp32(x, w, torch.float16)
    for i in range(3):
        x.normal_()
        x *= 10.0 ** (8 * i - 8)
        want = gradient_of_fp32(x, w, torch.float16)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
