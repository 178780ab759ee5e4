"""The bias's gradient of the linear layers: captured with its step, and its own derivative."""

import pytest
import torch

import gemv_int4_quantize_amd as w4

DEV = "cuda:0"
LAYERS = {"int4": (w4.w4a16_linear, lambda w: w4.quantize_pack(w, "rowwise")), "int8": (w4.w8a8_linear, lambda w: w4.quantize_int8(w)),
          "mxfp4": (w4.mxfp4_linear, lambda w: w4.quantize_mxfp4(w))}


def _randn(seed, *shape):
    return torch.randn(*shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", LAYERS)
@pytest.mark.parametrize("bdt", [torch.float32, torch.float16, torch.bfloat16, torch.float64])
@pytest.mark.parametrize("m,n,out_dtype", [(5, 64, None), (15, 2048, None), (16, 48, None), (2048, 1024, None), (4096, 96, torch.bfloat16), (8192, 256, None)])
def test_captured_step(kind, m, n, out_dtype, bdt):
    """Forward and backward in one graph, the bias's gradient with it, over several replays."""
    linear, make = LAYERS[kind]
    w = make(_randn(n, n, 256) * 0.05)
    odt = out_dtype or torch.float32
    x = _randn(m, m, 256).bfloat16().requires_grad_()
    bias = _randn(1, n).to(bdt).requires_grad_()
    gy = _randn(2, m, n).to(odt)

    def step(x, bias):
        y = linear(x, w, bias, out_dtype)
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
    half = {torch.float32: 2.0**-24, torch.float64: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}[bdt]
    for i in range(5):
        with torch.no_grad():
            x.copy_(_randn(10 + i, m, 256))
            bias.copy_(_randn(20 + i, n))
            gy.copy_(_randn(30 + i, m, n))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in out]
        plain = eager()
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1]) and got[2].dtype == plain[2].dtype == bdt, i
        # fp32 additions in any order, each off by at most half an ulp of a partial sum, and one rounding
        want, most = gy.double().sum(0), gy.double().abs().sum(0)
        for db in (got[2], plain[2]):
            assert ((db.double() - want).abs() <= most * (m * 2.0**-24) + want.abs() * half * 1.01).all(), i
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[2], got[2])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", LAYERS)
def test_types_and_strides(kind):
    """A bias of another type than the output's, an expanded gradient, one token, none."""
    linear, make = LAYERS[kind]
    n = 72
    w = make(_randn(3, n, 256) * 0.05)
    for m in (0, 1, 3, 300):
        for bdt in (torch.float32, torch.float16, torch.bfloat16, torch.float64):
            bias = torch.zeros(n, dtype=bdt, device=DEV, requires_grad=True)
            linear(_randn(4, m, 256), w, bias).sum().backward()
            assert bias.grad.dtype == bdt and (bias.grad == m).all()
    gy = torch.arange(n * 6, device=DEV).view(n, 2, 3).float().permute(1, 2, 0)  # columns apart
    x = _randn(5, 2, 3, 256)
    bias = torch.zeros(n, device=DEV, requires_grad=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = torch.autograd.grad(linear(x, w, bias), bias, gy)[0]
    graph.replay()
    bias = torch.zeros(n, device=DEV, requires_grad=True)
    linear(x, w, bias).backward(gy)
    assert torch.equal(bias.grad, gy.sum((0, 1))) and torch.equal(captured, bias.grad)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["int4", "int8"])  # (mxfp4's is differentiable once)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m", [7, 40])
def test_derivative_of_the_sum(kind, dtype, m):
    """The bias's gradient is linear in the output's: differentiated, it hands its gradient to every row."""
    linear, make = LAYERS[kind]
    w = make(_randn(6, 24, 256))
    x, h = _randn(7, m, 256), _randn(8, 24).to(dtype)

    def step():
        bias = torch.zeros(24, dtype=dtype, device=DEV, requires_grad=True)
        gy = ones.detach().clone().requires_grad_()
        (db,) = torch.autograd.grad(linear(x, w, bias, dtype), bias, gy, create_graph=True)
        return db, *torch.autograd.grad(db, gy, h)

    ones = torch.ones(m, 24, dtype=dtype, device=DEV)
    eager = step()
    eager = [t.detach().clone() for t in eager]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    graph.replay()
    torch.cuda.synchronize()
    for db, back in (eager, captured):
        assert (db == m).all() and back.dtype == dtype and torch.equal(back, h.expand(m, 24))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", LAYERS)
@pytest.mark.parametrize("n", [24, 2048])
def test_few_rows_agree(kind, n):
    """Sums of few rows have the bits of torch's in every layer, also where terms cancel."""
    linear, make = LAYERS[kind]
    w = make(_randn(9, n, 256))
    for m in (1, 2, 14, 15):
        gy = _randn(m, m, n)
        gy[-1] = -gy[:-1].double().sum(0).float()
        bias = torch.zeros(n, device=DEV, requires_grad=True)
        linear(_randn(1, m, 256), w, bias).backward(gy)
        assert torch.equal(bias.grad, gy.sum(0))
