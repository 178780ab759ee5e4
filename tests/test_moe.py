"""The mixture-of-experts layer on MXFP4 weights: refusals on the host, and on the GPU against the
formula in 64 bits over types, masks, ties and sizes."""

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
FLOATS = [torch.float32, torch.float16, torch.bfloat16]
INF = float("inf")


def _p(v=0x10000):  # an aligned address that is never dereferenced: every call below is refused
    return ctypes.c_void_p(v)


# ---------------------------------------------------------------- host only


def test_refusals():
    L = w4.lib()

    def moe(X=_p(), dt=2, ldx=64, T=3, z=_p(), zdt=0, ldl=8, E=8, top=2, W1=_p(), s1=_p(), W2=_p(), s2=_p(), H=64, F=96,
            out=_p(), ldo=64, ws=_p(), wsb=1 << 40):
        return L.mx4_moe(X, dt, ldx, T, z, zdt, ldl, E, top, 1, W1, s1, W2, s2, H, F, out, ldo, ws, wsb, None)

    assert moe(dt=3) == _lib.W4_ERR_INVALID
    assert moe(zdt=3) == _lib.W4_ERR_INVALID
    assert moe(T=-1) == _lib.W4_ERR_INVALID
    assert moe(E=0, top=0) == _lib.W4_ERR_INVALID
    assert moe(H=0) == _lib.W4_ERR_INVALID
    assert moe(F=0) == _lib.W4_ERR_INVALID
    assert moe(top=0) == _lib.W4_ERR_INVALID
    assert moe(top=9) == _lib.W4_ERR_INVALID
    assert moe(E=513, ldl=513) == _lib.W4_ERR_UNSUPPORTED
    assert moe(E=64, ldl=64, top=17) == _lib.W4_ERR_UNSUPPORTED
    assert moe(F=1 << 18) == _lib.W4_ERR_UNSUPPORTED
    assert moe(H=1 << 18, ldx=1 << 18, ldo=1 << 18) == _lib.W4_ERR_UNSUPPORTED
    assert moe(X=None) == _lib.W4_ERR_INVALID
    assert moe(z=None) == _lib.W4_ERR_INVALID
    assert moe(out=None) == _lib.W4_ERR_INVALID
    assert moe(W1=None) == _lib.W4_ERR_INVALID
    assert moe(s2=None) == _lib.W4_ERR_INVALID
    assert moe(ldx=63) == _lib.W4_ERR_INVALID
    assert moe(ldl=7) == _lib.W4_ERR_INVALID
    assert moe(ldo=63) == _lib.W4_ERR_INVALID
    assert moe(W2=_p(0x10008)) == _lib.W4_ERR_ALIGN
    assert moe(z=_p(0x10002)) == _lib.W4_ERR_ALIGN
    assert moe(ws=_p(0x10008)) == _lib.W4_ERR_ALIGN
    assert moe(T=0, X=None, z=None, out=None, W1=None) == _lib.W4_OK
    size = ctypes.c_size_t(0)
    assert L.mx4_moe_workspace_bytes(3, 8, 2, 64, 96, 2, ctypes.byref(size)) == 0 and size.value > 0
    assert moe(wsb=size.value - 1) == _lib.W4_ERR_RESOURCE and moe(ws=None, wsb=0) == _lib.W4_ERR_RESOURCE
    assert L.mx4_moe_workspace_bytes(0, 8, 2, 64, 96, 2, ctypes.byref(size)) == 0 and size.value == 0
    assert L.mx4_moe_workspace_bytes(3, 8, 2, 64, 96, 2, None) == _lib.W4_ERR_INVALID
    assert L.mx4_moe_workspace_bytes(3, 8, 9, 64, 96, 2, ctypes.byref(size)) == _lib.W4_ERR_INVALID
    # many tokens run 64 at a time in the workspace of 64
    assert L.mx4_moe_workspace_bytes(64, 8, 2, 64, 96, 2, ctypes.byref(size)) == 0
    at64 = size.value
    assert L.mx4_moe_workspace_bytes(5000, 8, 2, 64, 96, 2, ctypes.byref(size)) == 0 and size.value == at64


def _empty(rows, cols):
    p = (cols + 127) // 128 * 128
    return w4.MXFP4Rows(torch.zeros(rows, p // 2, dtype=torch.uint8), torch.zeros(rows, p // 32, dtype=torch.uint8), rows, cols)


def test_binding_refusals():
    w1, w2 = _empty(4 * 2 * 40, 64), _empty(4 * 64, 40)
    x, z = torch.zeros(2, 64), torch.zeros(2, 4)
    with pytest.raises(ValueError, match="HIP device"):
        w4.moe_mxfp4(x, z, w1, w2, 2)
    with pytest.raises(ValueError, match="need w1"):
        w4.moe_mxfp4(x, torch.zeros(2, 5), w1, w2, 2)
    with pytest.raises(ValueError, match="need w1"):
        w4.moe_mxfp4(torch.zeros(2, 65), z, w1, w2, 2)
    with pytest.raises(ValueError, match="need w1"):
        w4.moe_mxfp4(x, z, w1, _empty(4 * 63, 40), 2)
    with pytest.raises(ValueError, match="tokens"):
        w4.moe_mxfp4(x, torch.zeros(3, 4), w1, w2, 2)
    with pytest.raises(ValueError, match="2-D"):
        w4.moe_mxfp4(torch.zeros(64), z, w1, w2, 2)
    with pytest.raises(TypeError):
        w4.moe_mxfp4(x.double(), z, w1, w2, 2)
    with pytest.raises(ValueError, match="out must"):
        w4.moe_mxfp4(x, z, w1, w2, 2, out=torch.zeros(2, 63))
    with pytest.raises(ValueError, match="scales"):
        w4.moe_mxfp4(x, z, w1, w4.MXFP4Rows(w2.codes, w2.scales[:-1], w2.rows, w2.cols), 2)
    for a, b in ((x.clone().requires_grad_(), z), (x, z.clone().requires_grad_())):
        with pytest.raises(RuntimeError, match="no derivative"):
            w4.moe_mxfp4(a, b, w1, w2, 2)
    with pytest.raises(ValueError, match="same experts"):
        w4.MXFP4MoE(w1, _empty(4 * 63, 40), 2)
    with pytest.raises(ValueError, match="top_k"):
        w4.MXFP4MoE(w1, w2, 5)
    assert w4.MXFP4MoE(w1, w2, 4).experts == 4


# ---------------------------------------------------------------- GPU


def _experts(seed, E, H, F):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (w4.quantize_mxfp4(torch.randn(E * 2 * F, H, device=DEV, generator=g) * H**-0.5),
            w4.quantize_mxfp4(torch.randn(E * H, F, device=DEV, generator=g) * F**-0.5))


def _inputs(seed, T, E, H, dtype, zdtype, masked=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed + 1000)
    x = torch.randn(T, H, device=DEV, generator=g).to(dtype)
    z = torch.randn(T, E, device=DEV, generator=g) * 1.5
    if masked:
        z.masked_fill_(torch.rand(T, E, device=DEV, generator=g) < masked, -INF)
    return x, z.to(zdtype)


def _reference(x, z, w1, w2, top, renorm):
    """The layer in 64 bits and a bound of the kernels' error before the last rounding."""
    dtype = x.dtype
    T, H = x.shape
    E, F = z.shape[1], w2.cols
    parts, between = (3, 2.0**-24) if dtype == torch.float32 else (2 if dtype == torch.float16 else 1, 2.0**-16)
    z64, x64 = z.double().cpu().numpy(), x.double().cpu().numpy()
    v1 = w4.dequantize_mxfp4(w1, torch.float32).cpu().numpy().astype(np.float64).reshape(E, 2 * F, H)
    v2 = w4.dequantize_mxfp4(w2, torch.float32).cpu().numpy().astype(np.float64).reshape(E, H, F)
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        if np.isnan(z64[t]).any() or (z64[t] == INF).any():
            y[t] = np.nan
            continue
        order = sorted(range(E), key=lambda e: (-z64[t, e], e))[:top]
        order = [e for e in order if z64[t, e] > -INF]
        if not order:
            continue
        m = z64[t].max()
        total = np.exp(z64[t][order] - m).sum() if renorm else np.exp(z64[t] - m).sum()
        size = np.zeros(H)
        for e in order:
            u = v1[e] @ x64[t]
            # exact products of each part, sums in any order, each rounded or cut (2 EPS32)
            du = 2 * (parts * H + 2) * EPS32 * (np.abs(v1[e]) @ np.abs(x64[t]))
            g, up, dg, dup = u[:F], u[F:], du[:F], du[F:]
            w = np.exp(z64[t, e] - m) / total
            s = g / (1 + np.exp(-g))
            a = s * up * w
            # |silu'| <= 1.1; a few roundings each of exponential, quotient and products, the total's sum
            # and the logit's distance in fp32; then the parts
            rel = (2 * E + 24 + abs(z64[t, e] - m)) * EPS32
            da = w * (1.1 * dg * (np.abs(up) + dup) + np.abs(s) * dup) + rel * (np.abs(a) + w * 1.1 * dg * np.abs(up))
            da += between * (np.abs(a) + da) + 2.0**-130
            y[t] += v2[e] @ a
            tol[t] += np.abs(v2[e]) @ da
            size += np.abs(v2[e]) @ (np.abs(a) + da)
        tol[t] += 2 * (3 * F * len(order) + 32) * EPS32 * size
    return y, tol


def _check(got, x, z, w1, w2, top, renorm, what=""):
    y, tol = _reference(x, z, w1, w2, top, renorm)
    g = got.double().cpu().numpy()
    assert got.dtype == x.dtype and g.shape == y.shape
    nan = np.isnan(y)
    assert (np.isnan(g) == nan).all(), what
    bound = tol + HALF_ULP[x.dtype] * (np.abs(y) + tol) + TINY[x.dtype]
    bad = ~(np.abs(g - y) <= bound) & ~nan
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {np.abs(g - y)[bad].max():.3e}"


SIZES = [  # T, E, top, H, F
    (1, 1, 1, 1, 1), (1, 8, 2, 64, 96), (1, 128, 8, 256, 128), (2, 4, 4, 130, 33), (3, 20, 3, 1003, 700), (5, 8, 2, 512, 300),
    (15, 16, 2, 128, 257), (16, 60, 4, 200, 130), (17, 8, 3, 192, 129), (31, 64, 6, 320, 64), (33, 3, 2, 96, 96),
    (48, 32, 1, 384, 200), (64, 128, 8, 256, 64), (64, 2, 2, 72, 40), (7, 512, 16, 64, 32), (64, 512, 16, 64, 32), (4, 8, 2, 2048, 1408),
    (1, 8, 2, 96, 7000), (4, 16, 4, 160, 1100)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,top,H,F", SIZES)
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("renorm", [True, False])
def test_layer(T, E, top, H, F, dtype, renorm):
    w1, w2 = _experts(E + H, E, H, F)
    for zdtype in (torch.float32, dtype):
        x, z = _inputs(T, T, E, H, dtype, zdtype)
        got = w4.moe_mxfp4(x, z, w1, w2, top, renormalize=renorm)
        _check(got, x, z, w1, w2, top, renorm, f"{zdtype}")
        assert torch.equal(w4.moe_mxfp4(x, z, w1, w2, top, renormalize=renorm), got)  # the same bits again


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("renorm", [True, False])
def test_masks_and_ties(dtype, renorm):
    """Masked experts, fewer than top_k left, none left, equal logits, zeros of both signs, NaN and
    infinities, the type's lowest value as a mask."""
    T, E, top, H, F = 12, 70, 5, 96, 72
    w1, w2 = _experts(5, E, H, F)
    for zdtype in FLOATS:
        x, z = _inputs(3, T, E, H, dtype, zdtype, masked=0.4)
        z[1] = -INF
        z[2, 3:] = -INF  # three or fewer are left
        z[3, :69] = -INF
        z[4] = 0.5  # the first five
        z[5] = 0.0
        z[5, 1::2] = -0.0
        z[6] = torch.finfo(zdtype).min
        z[6, 7] = 2.0
        z[7, 9] = float("nan")
        z[8, 69] = INF
        z[9, 10:20] = 30.0
        z[10] = -INF
        z[10, 64] = -200.0
        got = w4.moe_mxfp4(x, z, w1, w2, top, renormalize=renorm)
        _check(got, x, z, w1, w2, top, renorm, f"{zdtype}")
        assert not got[1].any() and torch.isnan(got[7:9]).all() and torch.isfinite(got[[0, 2, 3, 4, 5, 6, 9, 10, 11]]).all()
    z = torch.full((40, E), -INF, device=DEV)  # no token reaches an expert
    x = torch.randn(40, H, device=DEV).to(dtype)
    for t in (1, 16, 40):
        assert not w4.moe_mxfp4(x[:t], z[:t], w1, w2, top, renormalize=renorm).any()


@pytest.mark.gpu
def test_masked_expert_is_not_run():
    """Weights of an expert that no token may reach do not matter, whatever they hold."""
    T, E, top, H, F = 6, 10, 4, 200, 150
    w1, w2 = _experts(9, E, H, F)
    for dtype in FLOATS:
        x, z = _inputs(4, T, E, H, dtype, torch.float32)
        z[:, 3] = -INF
        z[2, 4:] = -INF  # three left of four
        want = w4.moe_mxfp4(x, z, w1, w2, top)
        b1, b2 = w4.MXFP4Rows(w1.codes, w1.scales.clone(), w1.rows, H), w4.MXFP4Rows(w2.codes, w2.scales.clone(), w2.rows, F)
        b1.scales[3 * 2 * F:4 * 2 * F] = 255
        b2.scales[3 * H:4 * H] = 255
        assert torch.equal(w4.moe_mxfp4(x, z, b1, b2, top), want)
        # a NaN block of an expert reaches the tokens that run it, and its rows of the output alone
        b2.scales[5 * H + 17, 0] = 255
        got = w4.moe_mxfp4(x, z, b1, b2, top)
        runs = (z.argsort(dim=1, descending=True, stable=True)[:, :top] == 5) & (z[:, 5] > -INF)[:, None]
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[runs.any(1), 17] = True
        assert torch.equal(torch.isnan(got), hit) and torch.equal(got[~hit], want[~hit])
        b2.scales[5 * H + 17, 0] = 254  # values past bf16's range
        got = w4.moe_mxfp4(x, z, b1, b2, top)
        assert torch.isfinite(got[~hit]).all() and torch.equal(got[~hit], want[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
def test_whole_numbers(dtype):
    """Experts whose gate saturates: silu(64) is 64 in fp32, so the layer is exact in whole numbers and
    any misplaced column, row or exponent shows."""
    E, H, F, top = 12, 160, 96, 3
    g = torch.Generator(device=DEV).manual_seed(1)
    gate = torch.zeros(E, F, H, device=DEV)
    gate[:, :, 0] = 1.0
    up = torch.zeros(E, F, H, device=DEV)
    place = torch.randint(1, H, (E, F), device=DEV, generator=g)
    up.scatter_(2, place[:, :, None], 1.0)
    down = torch.randint(-2, 3, (E, H, F), device=DEV, generator=g).float()
    down[:, :, ::32] = 4.0
    w1, w2 = w4.quantize_mxfp4(torch.cat([gate, up], 1).flatten(0, 1)), w4.quantize_mxfp4(down.flatten(0, 1))
    assert torch.equal(w4.dequantize_mxfp4(w2).float(), down.flatten(0, 1))
    for T in (1, 5, 16, 23, 64):
        x = torch.randint(-1, 2, (T, H), device=DEV, generator=g).to(dtype)
        x[:, 0] = 64
        z = torch.zeros(T, E, device=DEV)
        chosen = torch.stack([torch.randperm(E, device=DEV, generator=g)[:top] for _ in range(T)])
        z.scatter_(1, chosen, 100.0)  # the others' share, e^-100, is 0 in fp32
        weight = torch.zeros(T, E, device=DEV).scatter_(1, chosen, 1.0)
        out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        for e in range(E):
            a = x.double()[:, place[e]] * 64
            out += weight[:, e:e + 1].double() * (a @ down[e].double().t())
        third = float(np.float32(1) / np.float32(3))
        # g_j = fp32(1/3); 64 * up * g_j keeps the leading bits of g_j (16, in fp32 all 24), the sum is fp32
        got = w4.moe_mxfp4(x, z, w1, w2, top).double()
        bits = 2.0**-23 if dtype == torch.float32 else 2.0**-16
        size = torch.zeros_like(out)
        for e in range(E):
            size += weight[:, e:e + 1].double() * ((x.double()[:, place[e]] * 64).abs() @ down[e].double().abs().t())
        tol = size * third * (bits + 2 * (3 * F * top + 8) * EPS32) + HALF_ULP[dtype] * out.abs() * 0.34
        assert ((got - out * third).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
def test_each_token_alone(dtype):
    """A token's result does not depend on which others are in the batch, beyond the order of sums."""
    T, E, top, H, F = 40, 16, 4, 256, 192
    w1, w2 = _experts(2, E, H, F)
    x, z = _inputs(8, T, E, H, dtype, torch.float32)
    whole = w4.moe_mxfp4(x, z, w1, w2, top)
    _check(whole, x, z, w1, w2, top, True)
    for t in (0, 17, 39):
        _check(w4.moe_mxfp4(x[t:t + 1], z[t:t + 1], w1, w2, top), x[t:t + 1], z[t:t + 1], w1, w2, top, True)
    many, mz = x.repeat(4, 1)[:147], z.repeat(4, 1)[:147]  # runs of 64
    y = w4.moe_mxfp4(many, mz, w1, w2, top)
    _check(y, many, mz, w1, w2, top, True)
    assert w4.moe_mxfp4(x[:0], z[:0], w1, w2, top).shape == (0, H)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
def test_strides_and_guards(dtype):
    """Rows of wider buffers for x, logits and the output; what lies around the output stays."""
    T, E, top, H, F = 9, 8, 2, 128, 64
    w1, w2 = _experts(4, E, H, F)
    for pad in (1, 8):
        x, z = _inputs(pad, T, E, H, dtype, dtype)
        want = w4.moe_mxfp4(x, z, w1, w2, top)
        wx = torch.full((T, H + pad), float("nan"), dtype=dtype, device=DEV)
        wz = torch.full((T, E + pad), float("nan"), dtype=dtype, device=DEV)
        wx[:, :H], wz[:, :E] = x, z
        guard = torch.full((T + 2, H + 2 * pad), 3.0, dtype=dtype, device=DEV)
        out = guard[1:-1, pad:-pad]
        assert w4.moe_mxfp4(wx[:, :H], wz[:, :E], w1, w2, top, out=out) is out
        assert torch.equal(out, want)
        assert (guard[0] == 3).all() and (guard[-1] == 3).all() and (guard[:, :pad] == 3).all() and (guard[:, -pad:] == 3).all()
        buf = torch.empty(T * H + 1, dtype=dtype, device=DEV)
        off = buf[1:].view(T, H)
        off.copy_(x)  # not 16-byte aligned
        assert torch.equal(w4.moe_mxfp4(off, z, w1, w2, top), want)
        assert torch.equal(w4.moe_mxfp4(x.t().contiguous().t(), z.t().contiguous().t(), w1, w2, top), want)


@pytest.mark.gpu
def test_special_activations():
    """NaN and infinities of a token's x stay in its row."""
    T, E, top, H, F = 6, 8, 2, 192, 64
    w1, w2 = _experts(6, E, H, F)
    for dtype in FLOATS:
        x, z = _inputs(2, T, E, H, dtype, torch.float32)
        want = w4.moe_mxfp4(x, z, w1, w2, top)
        x[1, 5], x[3, 7] = float("nan"), INF
        got = w4.moe_mxfp4(x, z, w1, w2, top)
        assert torch.isnan(got[1]).all() and not torch.isfinite(got[3]).any()
        keep = [0, 2, 4, 5]
        assert torch.equal(got[keep], want[keep])


@pytest.mark.gpu
def test_far_offsets():
    """Expert weights of more than 2^31 bytes: the first, the last and one across the border."""
    E, H, F, top = 128, 4096, 4224, 2
    g = torch.Generator(device=DEV).manual_seed(3)

    def rows(r, c):
        codes = torch.randint(0, 256, (r, c // 2), dtype=torch.uint8, device=DEV, generator=g)
        return w4.MXFP4Rows(codes, torch.full((r, c // 32), 121, dtype=torch.uint8, device=DEV), r, c)

    w1, w2 = rows(E * 2 * F, H), rows(E * H, F)
    assert w1.codes.numel() > 1 << 31
    few = [0, 62, 124, 127]

    def part(w, per):
        at = torch.cat([torch.arange(e * per, (e + 1) * per, device=DEV) for e in few])
        return w4.MXFP4Rows(w.codes[at], w.scales[at], len(few) * per, w.cols)

    p1, p2 = part(w1, 2 * F), part(w2, H)
    x = torch.randn(4, H, device=DEV).bfloat16() * 0.02
    z = torch.full((4, E), -INF, device=DEV)
    z[:, few] = torch.randn(4, 4, device=DEV)
    got, want = w4.moe_mxfp4(x, z, w1, w2, top), w4.moe_mxfp4(x, z[:, few].contiguous(), p1, p2, top)
    torch.testing.assert_close(got.float(), want.float(), rtol=2.0**-7, atol=1e-3 * want.float().abs().max().item())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_streams_and_graph_replays(T, dtype):
    E, top, H, F = 16, 4, 256, 384
    w1, w2 = _experts(7, E, H, F)
    x, z = _inputs(1, T, E, H, dtype, torch.float32)
    want = w4.moe_mxfp4(x, z, w1, w2, top)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:  # two calls at once
        with torch.cuda.stream(s):
            for _ in range(4):
                got.append(w4.moe_mxfp4(x, z, w1, w2, top))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = w4.moe_mxfp4(x, z, w1, w2, top)
        y2 = w4.moe_mxfp4(y, z, w1, w2, top)
    for i in range(3):
        nx, nz = _inputs(50 + i, T, E, H, dtype, torch.float32, masked=0.2 * i)
        x.copy_(nx)
        z.copy_(nz)
        want = w4.moe_mxfp4(x, z, w1, w2, top)
        want2 = w4.moe_mxfp4(want, z, w1, w2, top)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(y2, want2)


@pytest.mark.gpu
def test_module():
    E, H, F = 6, 96, 80
    gate_up, down = torch.randn(E, 2 * F, H, device=DEV) * 0.1, torch.randn(E, H, F, device=DEV) * 0.1
    layer = w4.MXFP4MoE.from_weight(gate_up, down, 2, renormalize=False)
    assert layer.experts == E
    x, z = torch.randn(2, 3, H, device=DEV).bfloat16(), torch.randn(2, 3, E, device=DEV)
    y = layer(x, z)
    assert y.shape == x.shape and y.dtype == x.dtype
    assert torch.equal(y.view(6, H), w4.moe_mxfp4(x.view(6, H), z.view(6, E), layer.w1, layer.w2, 2, renormalize=False))


@pytest.mark.gpu
def test_decoding_step_of_a_block():
    """The operators together, as a decoding step runs them: a fused projection, a router's logits, the
    experts, a head, and the scores of its tokens."""
    T, H, F, E, V = 6, 256, 192, 16, 515
    g = torch.Generator(device=DEV).manual_seed(11)

    def rand(*shape):
        return torch.randn(*shape, device=DEV, generator=g) * shape[-1] ** -0.5

    inner = w4.MXFP4Linear.from_weight(rand(H, H), out_dtype=torch.bfloat16)
    router = w4.MXFP4Linear.from_weight(rand(E, H))
    moe = w4.MXFP4MoE.from_weight(rand(E, 2 * F, H), rand(E, H, F), 4)
    head = w4.MXFP4Linear.from_weight(rand(V, H), out_dtype=torch.bfloat16)
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    with torch.no_grad():
        h = inner(x)
        z = router(h)
        y = moe(h, z)
        s = w4.token_logprobs(head(y), torch.zeros(T, dtype=torch.int64, device=DEV), top=3)
    _check(y, h, z, moe.w1, moe.w2, 4, True)
    q = w4.dequantize_mxfp4(w4.quantize_mxfp4(y), torch.float32).double()
    logits = q @ w4.dequantize_mxfp4(head.w, torch.float32).double().t()
    ref = torch.log_softmax(logits, 1)
    # bf16 logits: half a step of each of two logits
    worst = 2 * logits.abs().max().item() * 2.0**-8 + 1e-4
    assert ((s.top_logprobs.double() - ref.gather(1, s.top_ids)).abs() <= worst).all()
    # and one of training through the frozen layers
    a = x.clone().requires_grad_()
    t = torch.randint(V, (T,), device=DEV, generator=g)
    (-w4.token_logprobs(head(inner(a)), t).logprobs.mean()).backward()
    with torch.no_grad():
        mid = inner(x)
        z = head(mid).double()
    dz = (torch.softmax(z, 1) - torch.nn.functional.one_hot(t, V)) / T
    wh, wi = (w4.dequantize_mxfp4(m.w, torch.float32).double() for m in (head, inner))
    d1 = dz @ wh
    ref = d1 @ wi
    # dz, dmid and dx each rounded to bf16 (2^-8), fp32 sums below
    step = 2.0**-8 + 2.0**-13
    e1 = (dz.abs() @ wh.abs()) * step + d1.abs() * step
    bound = e1 @ wi.abs() + ref.abs() * step + (d1.abs() @ wi.abs()) * 2.0**-13 + 1e-12
    assert ((a.grad.double() - ref).abs() <= bound).all()
