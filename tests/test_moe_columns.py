"""The experts' layer where experts have many tokens (sixteen columns a product), on contractions of several
units, and what it keeps of the activations between its two products."""

import pytest
import torch

import gemv_int4_quantize_amd as w4
from test_moe import DEV, EPS32, FLOATS, HALF_ULP, TINY, _experts, _inputs

INF = float("inf")


def _part(w, first, rows):
    return w4.dequantize_mxfp4(w4.MXFP4Rows(w.codes[first:first + rows], w.scales[first:first + rows], rows, w.cols), torch.float32).double()


def _expected(x, z, w1, w2, top, renorm):
    """The layer in 64 bits and a bound of the kernels' error before the last rounding, an expert at a
    time."""
    dtype, (T, H) = x.dtype, x.shape
    E, F = z.shape[1], w2.cols
    parts = {torch.float32: 3, torch.float16: 2, torch.bfloat16: 1}[dtype]
    z, x = z.double(), x.double()
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]
    chosen = torch.zeros(T, E, dtype=torch.bool, device=DEV).scatter_(1, order, True) & (z > -INF)
    m = z.amax(1, keepdim=True).clamp(min=-1e300)
    p = torch.exp(z - m)
    total = torch.where(chosen | (not renorm), p, 0.0).sum(1, keepdim=True)
    weight = torch.where(chosen, p / torch.where(total > 0, total, 1.0), 0.0)
    y, tol, size = (torch.zeros(T, H, dtype=torch.float64, device=DEV) for _ in range(3))
    for e in range(E):
        t = torch.nonzero(chosen[:, e]).flatten()
        if not len(t):
            continue
        a1, a2 = _part(w1, e * 2 * F, 2 * F), _part(w2, e * H, H)
        u = x[t] @ a1.t()
        # exact products of each part, sums in any order, each rounded or cut (2 EPS32)
        du = 2 * (parts * H + 2) * EPS32 * (x[t].abs() @ a1.abs().t())
        g, up, dg, dup = u[:, :F], u[:, F:], du[:, :F], du[:, F:]
        w = weight[t, e][:, None]
        s = g / (1 + torch.exp(-g))
        a = s * up * w
        # |silu'| <= 1.1; a few roundings each of exponential, quotient and products, the total's sum and
        # the logit's distance in fp32; between the products all of fp32's bits
        rel = (2 * E + 24 + (z[t, e][:, None] - m[t]).abs()) * EPS32
        da = w * (1.1 * dg * (up.abs() + dup) + s.abs() * dup) + rel * (a.abs() + w * 1.1 * dg * up.abs()) + 2.0**-130
        y[t] += a @ a2.t()
        tol[t] += da @ a2.abs().t()
        size[t] += (a.abs() + da) @ a2.abs().t()
    return y, tol + 2 * (3 * F * top + 32) * EPS32 * size


def _check(got, *args):
    y, tol = _expected(*args)
    dtype = args[0].dtype
    g = got.double()
    assert got.dtype == dtype and g.shape == y.shape
    bad = ~((g - y).abs() <= tol + HALF_ULP[dtype] * (y.abs() + tol) + TINY[dtype])
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst {(g - y).abs()[bad].max().item():.3e}"


# T, E, top, H, F with T > 4 and T top > 3 E: waves with several units and a last one that is half a unit; more
# items than workgroups; waves of the second launch with several units of several experts, at both ring
# depths; to four tokens an expert; a batch whose tokens all agree, and experts without any
WIDE = [(20, 4, 2, 2500, 700), (33, 8, 4, 1300, 1100), (20, 8, 3, 4100, 1100), (64, 8, 3, 4100, 1100), (64, 4, 1, 1150, 2300),
        (7, 2, 1, 900, 1410), (37, 5, 5, 260, 520), (13, 8, 2, 2100, 1300), (30, 16, 2, 700, 520)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,top,H,F", WIDE)
@pytest.mark.parametrize("dtype", FLOATS)
def test_many_tokens_an_expert(T, E, top, H, F, dtype):
    assert T > 4 and T * top > 3 * E
    w1, w2 = _experts(E + H, E, H, F)
    for renorm, masked in ((True, 0.0), (False, 0.3)):
        x, z = _inputs(T + H, T, E, H, dtype, torch.float32 if renorm else dtype, masked)
        got = w4.moe_mxfp4(x, z, w1, w2, top, renormalize=renorm)
        _check(got, x, z, w1, w2, top, renorm)
        assert torch.equal(w4.moe_mxfp4(x, z, w1, w2, top, renormalize=renorm), got)
    z = z[:1].expand(T, E).contiguous()  # every token to the same experts
    z[:, E - 1] = -INF
    _check(w4.moe_mxfp4(x, z, w1, w2, top), x, z, w1, w2, top, True)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 40, 64])
def test_agreeing_tokens_on_few_columns(T):
    """Tokens that all choose the same of many experts: more of them than a product's four columns."""
    E, top, H, F = 64, 2, 1290, 390
    assert T * top <= 3 * E
    w1, w2 = _experts(T, E, H, F)
    for dtype in FLOATS:
        x, z = _inputs(T, T, E, H, dtype, torch.float32)
        z = z[:1].expand(T, E).contiguous()
        _check(w4.moe_mxfp4(x, z, w1, w2, top), x, z, w1, w2, top, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,E,H,F", [(1, 1, 64, 32), (1, 1, 1100, 2100), (4, 2, 2100, 300), (16, 64, 200, 40), (16, 2, 1300, 300),
                                     (8, 64, 96, 2000), (38, 64, 96, 40), (39, 64, 96, 40),
                                     (64, 3, 96, 64)])
def test_nothing_is_lost_between_the_products(T, E, H, F, dtype):
    """Differences of nearly equal activations come out whole: silu(64) is 64 in fp32, so that
    g a = 64 (1 + 2^-8 + 2^-j) and 64 (1 + 2^-8) for the columns that the down projection subtracts, both
    exact in fp32; 64 2^-j is left for every j down to fp32's last bit."""
    gate_up, down = torch.zeros(E, 2 * F, H, device=DEV), torch.zeros(E, H, F, device=DEV)
    one, more, small, last = H // 2, H - 3, H - 2, H - 1
    gate_up[:, :F, 0] = 1.0
    gate_up[:, F:, one] = gate_up[:, F:, more] = 1.0
    gate_up[:, F, small] = 1.0  # the first activation has the small number too
    down[:, :, 0], down[:, :, F - 1] = 1.0, -1.0
    down[:, last] = -down[:, last]
    w1, w2 = w4.quantize_mxfp4(gate_up.flatten(0, 1)), w4.quantize_mxfp4(down.flatten(0, 1))
    j = torch.arange(T, device=DEV) % 7 + 17 if T > 1 else torch.tensor([19], device=DEV)
    x = torch.zeros(T, H, device=DEV)
    x[:, 0], x[:, one], x[:, more], x[:, small] = 64.0, 1.0, 2.0**-8, torch.exp2(-j.float())
    z = torch.full((T, E), -INF, device=DEV)
    z[torch.arange(T, device=DEV), torch.arange(T, device=DEV) % E] = 0.5
    y = w4.moe_mxfp4(x.to(dtype), z, w1, w2, 1).double()
    want = torch.exp2(6.0 - j.double())[:, None].repeat(1, H)
    want[:, last] *= -1
    assert torch.equal(y, want)
