"""Few float tokens of the MXFP4 product where a workgroup goes through several groups of channels, its waves
through several units of each."""

import pytest
import torch

import gemv_int4_quantize_amd as w4
from test_mxfp4 import DEV, FLOATS

# groups of 32 channels past two for every CU (N >= 16384): up to four tokens and up to eight, up to 4096
# columns and more, each with at least three groups a workgroup and an odd rest; and groups of 16
WALKS = [(1, 50021, 4090), (4, 50021, 4000), (1, 50021, 8010), (4, 50021, 8100), (3, 40001, 14900), (6, 50021, 1100), (8, 50021, 4000),
         (5, 50021, 6000), (8, 16411, 2100), (4, 16000, 9000), (2, 16383, 4100), (7, 16001, 4500), (8, 16383, 1030), (1, 12291, 16300)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", WALKS)
@pytest.mark.parametrize("dtype", FLOATS)
def test_walk_over_groups(m, n, k, dtype):
    """Whole numbers, so that every sum is exact: tokens whose blocks reach 4 keep the power, weights of random
    codes at two powers.  Terms are multiples of 1/4 up to 48."""
    assert w4.mxfp4_kernel_for(m, n, k) == "mx4_decode_fused"
    assert 4 * 48 * k < 1 << 24
    g = torch.Generator(device=DEV).manual_seed(m * 31 + n)
    p = (k + 127) // 128 * 128
    codes = torch.randint(0, 256, (n, p // 2), dtype=torch.uint8, device=DEV, generator=g)
    codes[:, (k + 1) // 2:] = 0
    if k % 2:
        codes[:, k // 2] &= 15
    w = w4.MXFP4Rows(codes, torch.randint(127, 129, (n, p // 32), dtype=torch.uint8, device=DEV, generator=g), n, k)
    x = torch.randint(-4, 5, (m, k), device=DEV, generator=g) * 0.5
    x[:, ::32] = 4.0
    x = x.to(dtype)
    bias = torch.randint(-9, 10, (n,), device=DEV, generator=g).float()
    want = torch.empty(m, n, dtype=torch.float64, device=DEV)
    for c in range(0, n, 8192):
        part = w4.MXFP4Rows(w.codes[c:c + 8192], w.scales[c:c + 8192], min(8192, n - c), k)
        want[:, c:c + 8192] = x.double() @ w4.dequantize_mxfp4(part, torch.float32).double().t()
    want += bias.double()
    assert torch.equal(w4.mm_mxfp4(x, w, bias=bias).double(), want)
    outs = [torch.full((m + 1, c), 5.0, device=DEV) for c in (33, n - 33)]
    w4.mm_mxfp4_split(x, w, [o[:m] for o in outs], bias=bias)
    assert torch.equal(torch.cat([o[:m] for o in outs], 1).double(), want) and all((o[m] == 5).all() for o in outs)


@pytest.mark.gpu
@pytest.mark.parametrize("k", [100, 300, 640, 1555, 3900])
@pytest.mark.parametrize("m", [2, 3, 5, 8])
def test_tokens_of_an_odd_number_of_pieces(m, k):
    """Rows of an odd multiple of 128 columns, once padded: each token's exponents meet its own codes."""
    n = 70
    g = torch.Generator(device=DEV).manual_seed(k + m)
    w = w4.quantize_mxfp4(torch.randint(-6, 7, (n, k), device=DEV, generator=g).float())
    x = torch.randint(-2, 3, (m, k), device=DEV, generator=g).float()
    x[:, ::32] = 4.0
    blocks = (k + 31) // 32
    power = torch.randint(-3, 4, (m, blocks), device=DEV, generator=g).float()
    x = x * torch.exp2(power).repeat_interleave(32, 1)[:, :k]
    q = w4.quantize_mxfp4(x)
    assert torch.equal(w4.dequantize_mxfp4(q, torch.float32), x)
    want = x.double() @ w4.dequantize_mxfp4(w, torch.float32).double().t()
    assert torch.equal(w4.mm_mxfp4(x, w).double(), want) and torch.equal(w4.mm_mxfp4(q, w).double(), want)


def test_long_rows_of_few_channels_are_split():
    """The few-token kernel does not split a row: where it would leave half of the CUs idle over a long one,
    tiles that split it run, and the workspace they ask for is reported."""
    import ctypes

    L = w4.lib()

    def kernel(m, n, k):
        return L.mx4_kernel(m, n, k, -1).decode()

    for m, n, k in ((16, 512, 65536), (32, 512, 65536), (32, 2048, 32768), (17, 100, 20480), (4, 2048, 40960), (2, 512, 65536)):
        assert "splitk" in kernel(m, n, k), (m, n, k)
        for xdt in (-1, 2):
            size = ctypes.c_size_t(0)
            assert L.mx4_workspace_bytes(m, n, k, xdt, ctypes.byref(size)) == 0
            assert size.value >= 2 * m * n * 4 + (0 if xdt < 0 else m * k * 17 // 32)
    for m, n, k in ((16, 512, 32768), (32, 512, 16384), (32, 2049, 65536), (16, 4096, 262144), (3, 128, 4096), (32, 128, 4096)):
        assert kernel(m, n, k) == "mx4_few", (m, n, k)
    assert kernel(1, 512, 40960) == "mx4_decode"


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(16, 512, 65500), (32, 500, 20500), (3, 40, 40961), (2, 100, 30001), (31, 2048, 18433), (17, 33, 18432),
                                   (1, 70, 60001), (8, 512, 36864), (9, 17, 36865)])
def test_long_rows(m, n, k):
    """Whole numbers of both kinds of tokens on both sides of the rule: |sum| <= 36 k, in quarters."""
    assert 4 * 36 * k < 1 << 24
    g = torch.Generator(device=DEV).manual_seed(m + n)

    def rows(r):
        c = torch.randint(0, 256, (r, (k + 127) // 128 * 64), dtype=torch.uint8, device=DEV, generator=g)
        c[:, (k + 1) // 2:] = 0
        if k % 2:
            c[:, k // 2] &= 15
        return w4.MXFP4Rows(c, torch.full((r, (k + 127) // 128 * 4), 127, dtype=torch.uint8, device=DEV), r, k)

    w = rows(n)
    x = w4.dequantize_mxfp4(rows(m), torch.float32)
    x[:, ::32] = 6.0  # blocks whose largest magnitude is 6 keep the power
    a = w4.quantize_mxfp4(x)
    assert torch.equal(w4.dequantize_mxfp4(a, torch.float32), x)
    want = x.double() @ w4.dequantize_mxfp4(w, torch.float32).double().t()
    for t in (a, x, x.bfloat16(), x.half()):
        assert torch.equal(w4.mm_mxfp4(t, w).double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1, 33, 130, 300, 1100])
def test_scales_past_the_last_column(k):
    """Blocks of nothing but padding may hold any scale but NaN's; the quantizer's are 0."""
    g = torch.Generator(device=DEV).manual_seed(k)
    n, blocks = 40, (k + 31) // 32
    w = w4.quantize_mxfp4(torch.randn(n, k, device=DEV, generator=g))
    x = torch.randn(70, k, device=DEV, generator=g).bfloat16()
    a = w4.quantize_mxfp4(x)
    assert not w.scales[:, blocks:].any() and not a.scales[:, blocks:].any()
    dirty = [w4.MXFP4Rows(r.codes, r.scales.clone(), r.rows, k) for r in (w, a)]
    for r in dirty:
        r.scales[:, blocks:] = torch.randint(1, 255, r.scales[:, blocks:].shape, dtype=torch.uint8, device=DEV, generator=g)
        assert torch.equal(w4.dequantize_mxfp4(r), w4.dequantize_mxfp4(w if r.rows == n else a))
    for m in (1, 3, 8, 20, 70):
        want = w4.mm_mxfp4(x[:m], w)
        some = w4.MXFP4Rows(dirty[1].codes[:m], dirty[1].scales[:m], m, k)
        assert torch.equal(w4.mm_mxfp4(x[:m], dirty[0]), want) and torch.equal(w4.mm_mxfp4(some, dirty[0]), w4.mm_mxfp4(some, w))
    dy = torch.randn(9, n, device=DEV, generator=g)
    assert torch.equal(w4.mm_mxfp4_t(dy, dirty[0]), w4.mm_mxfp4_t(dy, w))
    w1 = w4.quantize_mxfp4(torch.randn(2 * 2 * 24, k, device=DEV, generator=g))  # two experts, k -> 24 -> k
    w2 = w4.quantize_mxfp4(torch.randn(2 * k, 24, device=DEV, generator=g))
    z = torch.randn(6, 2, device=DEV, generator=g)
    want = w4.moe_mxfp4(x[:6], z, w1, w2, 1)
    w1.scales[:, blocks:], w2.scales[:, 1:] = 254, 254
    assert torch.equal(w4.moe_mxfp4(x[:6], z, w1, w2, 1), want)
