"""Scores of given tokens: refusals on the host; on the GPU against 64-bit arithmetic, with
the rows where a softmax goes wrong, and the gradient against its formula and differences."""

import ctypes
import math

import pytest
import torch

import gemv_int4_quantize_amd as w4
from gemv_int4_quantize_amd import _lib

DEV = "cuda:0"
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
HALF_ULP = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float32: 2.0**-149, torch.float16: 2.0**-24, torch.bfloat16: 2.0**-133}


# ---------------------------------------------------------------- host only


def _p(v=0x10000):
    return ctypes.c_void_p(v)


def test_refusals():
    L = w4.lib()

    def fwd(z=_p(), dt=0, M=4, V=100, ld=100, t=_p(), temp=1.0, top=0, lp=_p(), top_lp=_p(), ids=_p()):
        return L.tok_logprobs(z, dt, M, V, ld, t, -100, temp, top, lp, _p(), _p(), top_lp, ids, _p(), 1 << 40, None)

    assert fwd(z=None) == _lib.W4_ERR_INVALID
    assert fwd(dt=3) == _lib.W4_ERR_INVALID
    assert fwd(M=-1) == _lib.W4_ERR_INVALID
    assert fwd(V=0) == _lib.W4_ERR_INVALID
    assert fwd(ld=99) == _lib.W4_ERR_INVALID
    assert fwd(t=None) == _lib.W4_ERR_INVALID
    assert fwd(lp=None) == _lib.W4_ERR_INVALID
    assert fwd(top=65) == _lib.W4_ERR_INVALID
    assert fwd(top=-1) == _lib.W4_ERR_INVALID
    assert fwd(V=10, top=11) == _lib.W4_ERR_INVALID
    assert fwd(top=3, ids=None) == _lib.W4_ERR_INVALID
    assert fwd(V=1 << 31, ld=1 << 31) == _lib.W4_ERR_UNSUPPORTED
    for temp in (0.0, -1.0, math.nan, math.inf, 1e-39):
        assert fwd(temp=temp) == _lib.W4_ERR_INVALID, temp
    assert fwd(z=_p(0x10002)) == _lib.W4_ERR_ALIGN
    assert fwd(t=_p(0x10004)) == _lib.W4_ERR_ALIGN
    assert fwd(M=0, z=None) == _lib.W4_OK

    def bwd(z=_p(), stats=_p(), ids=_p(), a=None, top=0, dz=_p(0x20000), ldd=100):
        return L.tok_logprobs_grad(z, 0, 4, 100, 100, _p(), -100, 1.0, top, stats, _p(), ids, None, None, a, dz, ldd, None)

    assert bwd(stats=None) == _lib.W4_ERR_INVALID
    assert bwd(dz=None) == _lib.W4_ERR_INVALID
    assert bwd(ldd=99) == _lib.W4_ERR_INVALID
    assert bwd(top=2, a=_p(), ids=None) == _lib.W4_ERR_INVALID
    assert bwd(dz=_p(), ldd=104) == _lib.W4_ERR_INVALID  # in place with another stride


def test_binding_refusals():
    z = torch.zeros(3, 10)
    with pytest.raises(ValueError, match="HIP device"):
        w4.token_logprobs(z, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="targets"):
        w4.token_logprobs(z, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="targets"):
        w4.token_logprobs(z, torch.zeros(3))
    with pytest.raises(TypeError):
        w4.token_logprobs(z.double(), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="2-D"):
        w4.token_logprobs(z[0], torch.zeros(3, dtype=torch.int64))

    def grad(t=torch.zeros(3, dtype=torch.int64), stats=torch.zeros(3, 2), ent=torch.zeros(3),
             ids=torch.zeros(3, 4, dtype=torch.int64), g=None, a=None, out=None):
        w4.token_logprobs_grad(z, t, stats, ent, ids, g, None, a, out=out)

    for bad in (dict(t=torch.zeros(2, dtype=torch.int64)), dict(stats=torch.zeros(3, 3)), dict(ent=torch.zeros(3).double()),
                dict(ids=torch.zeros(3, 4, dtype=torch.int32)), dict(ids=torch.zeros(3, dtype=torch.int64)),
                dict(g=torch.zeros(4)), dict(a=torch.zeros(3, 5)), dict(out=torch.zeros(3, 11)), dict()):
        with pytest.raises(ValueError):  # the last: not on a device
            grad(**bad)


# ---------------------------------------------------------------- GPU


def _logits(seed, m, v, dtype, pad=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(m, v, generator=g) * spread
    z[:, :: max(1, v // 7)] += 5.0
    wide = torch.full((m, v + pad), float("nan"))
    wide[:, :v] = z
    t = torch.randint(0, v, (m,), generator=g)
    return wide.to(dtype).to(DEV)[:, :v], t.to(DEV)


def _reference(z, t, top, temperature, ignore=-100):
    """The definition in 64 bits (temperature's reciprocal as the fp32 it is)."""
    inv = torch.tensor(1.0 / temperature, dtype=torch.float32).double().item()
    bad = ~(z < math.inf).all(1)
    empty = (z == -math.inf).all(1)
    u = (z.double() - torch.where(empty, torch.zeros_like(z[:, 0]), z.amax(1)).double()[:, None]) * inv
    lse = torch.logsumexp(torch.where(empty[:, None], torch.zeros_like(u), u), 1)
    logp = u - lse[:, None]
    p = torch.exp(logp)
    ent = -(torch.where(p > 0, p * logp, torch.zeros_like(p))).sum(1)
    lp = torch.full_like(lse, math.nan)
    inside = (t >= 0) & (t < z.shape[1])
    lp[inside] = logp[inside].gather(1, t[inside, None]).squeeze(1)
    ids = torch.sort(z.double(), dim=1, descending=True, stable=True).indices[:, :top]
    top_lp = logp.gather(1, ids)
    lp[empty & inside] = -math.inf
    top_lp[empty] = -math.inf
    ent[empty] = 0
    lp[bad], ent[bad], top_lp[bad], ids[bad] = math.nan, math.nan, math.nan, -1
    lp[t == ignore] = 0
    return lp, ent, top_lp, ids, p, logp, empty, bad


def _tol(z, temperature):
    """Absolute error of a log probability, for logits within 60 of their maximum (or so far below it
    that they are compared as infinities or relative to their size): fp32 roundings of d and the
    sum, whose terms carry the rounding of their exponents and are added in runs of at most
    v / 64 and a tree."""
    v = z.shape[1]
    return 2.0**-24 * (6 * 60 / temperature + v / 64 + 60) + 2.0**-20


def _same(x, ref, tol, what):
    x, ref = x.double().cpu(), ref.float().double().cpu()  # the outputs are fp32: so is their range
    assert torch.equal(torch.isnan(x), torch.isnan(ref)), what
    inf = torch.isinf(ref)
    assert torch.equal(torch.where(inf, x, torch.zeros_like(x)), torch.where(inf, ref, torch.zeros_like(ref))), what
    d = torch.where(torch.isfinite(ref), (x - ref).abs(), torch.zeros_like(ref))
    tol = tol + torch.where(torch.isfinite(ref), 2.0**-22 * ref.abs(), torch.zeros_like(ref))
    assert (d <= tol).all(), f"{what}: {(d - tol).max().item():.3e} over the tolerance"


def _check(z, t, top, temperature, ignore=-100):
    r = w4.token_logprobs(z, t, top=top, temperature=temperature, ignore_index=ignore)
    lp, ent, top_lp, ids, *_ = _reference(z, t.long(), top, temperature, ignore)
    tol = _tol(z, temperature)
    _same(r.logprobs, lp, tol, "logprobs")
    # entropy is a mean of -log p: the tolerance of log p, and the relative error of p on terms up to log V
    _same(r.entropy, ent, tol * (2 + math.log(z.shape[1])), "entropy")
    _same(r.top_logprobs, top_lp, tol, "top")
    assert torch.equal(r.top_ids, ids)


CASES = [(1, 1, 1, 0), (2, 2, 2, 0), (3, 5, 0, 1), (1, 64, 64, 0), (4, 100, 7, 0), (5, 1000, 20, 3), (3, 4097, 1, 0),
         (2, 32003, 20, 5), (1, 128256, 5, 0), (9, 50257, 64, 1), (300, 515, 8, 0), (1200, 2048, 5, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,v,top,pad", CASES)
def test_scores(m, v, top, pad, dtype):
    z, t = _logits(m + v, m, v, dtype, pad)
    _check(z, t, top, 1.0)
    _check(z, t, min(top, 3), 0.7)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,v", [(12, 333), (12, 40000), (600, 3001)])
def test_special_rows(m, v, dtype):
    z, t = _logits(v, m, v, dtype)
    lowest = torch.finfo(dtype).min
    z[0] = -math.inf  # nothing left
    z[1, 3] = math.nan
    z[2, v - 1] = math.inf
    z[3] = lowest  # a mask of the type's lowest value, over everything
    z[4, 5:] = -math.inf  # five left, fewer than the alternatives
    z[5] = -math.inf
    z[5, v // 2] = 1.0  # one left
    z[6] = 2.0  # all equal: ties to the lowest ids
    z[7, ::2] = lowest
    z[8, t[8]] = -math.inf  # the target is masked
    z[9] = torch.where(torch.arange(v, device=DEV) % 3 == 0, -0.0, 0.0).to(dtype)  # zeros of both signs are equal
    t[10] = -100
    t[11] = v
    _check(z, t, 8, 1.0)
    t[11] = -1
    _check(z, t.to(torch.int32), 8, 1.3)
    _check(z, t, 8, 0.5, ignore=int(t[3]))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 7, 700])
def test_ordered_rows(m):
    """Rows that rise, fall, or hold one value: the alternatives lie together or at either end."""
    v = 9001
    ramp = torch.arange(v, device=DEV).float() * 0.01
    for row in (ramp, -ramp, torch.zeros_like(ramp), torch.where(ramp < 1, 7.0, ramp * 0)):
        z = row.expand(m, v).contiguous()
        _check(z, torch.full((m,), v - 1, device=DEV), 64, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 1100])
def test_large_logits_in_few_places(m):
    """Most of the large logits of a row where few threads read them: runs of eight logits every
    2048, more of them above any group's maximum than are ranked at a time."""
    v = 130001
    z = torch.arange(v, device=DEV).float().mul_(1e-5)
    j = torch.arange(v, device=DEV)
    few = (j % 2048) < 8 * 12
    z = torch.where(few, 50.0 + z, z)
    z = z[torch.arange(v, device=DEV)].expand(m, v).contiguous()
    t = torch.full((m,), 7, device=DEV)
    r = w4.token_logprobs(z, t, top=64)
    ids = torch.sort(z[0].double(), descending=True, stable=True).indices[:64]
    assert (r.top_ids == ids).all()
    assert torch.allclose(r.logprobs, torch.log_softmax(z[:1].double(), 1)[0, 7].float().expand(m), atol=1e-4)


@pytest.mark.gpu
def test_temperature_overflow():
    """Logits that the temperature would take past fp32 are compared before it is applied."""
    z = torch.zeros(2, 10, device=DEV)
    z[0, 4] = 1e38
    r = w4.token_logprobs(z, torch.tensor([4, 0], device=DEV), top=2, temperature=1e-3)
    assert r.logprobs[0] == 0 and r.entropy[0] == 0 and r.top_ids[0, 0] == 4
    assert r.top_logprobs[0, 1] == -math.inf and abs(r.logprobs[1].item() + math.log(10)) < 1e-6


@pytest.mark.gpu
def test_far_offsets():
    """Rows more than 2^31 elements apart from the first."""
    ld, v = (1 << 30) + 5, 3001
    big = torch.empty(2 * ld + v, dtype=torch.float16, device=DEV)
    z = big.as_strided((3, v), (ld, 1))
    src, t = _logits(3, 3, v, torch.float16)
    z.copy_(src)
    _check(z, t, 5, 1.0)
    r = w4.token_logprobs(z, t)
    ids = torch.empty(3, 0, dtype=torch.int64, device=DEV)
    g = torch.ones(3, device=DEV)
    want = w4.token_logprobs_grad(src.contiguous(), t, r.stats, r.entropy, ids, g)
    got = w4.token_logprobs_grad(z, t, r.stats, r.entropy, ids, g, out=z)  # in place
    assert torch.equal(got, want)


def _gradient(z, t, top, temperature, g, h, a, ignore=-100):
    lp, ent, top_lp, ids, p, logp, empty, bad = _reference(z, t.long(), top, temperature, ignore)
    inv = torch.tensor(1.0 / temperature, dtype=torch.float32).double().item()
    m, v = z.shape
    inside = (t >= 0) & (t < v) & (t != ignore)
    g = torch.where(inside, g.double(), torch.zeros(m, dtype=torch.float64, device=DEV))
    total = g + a.double().sum(1)
    safe = torch.where(p > 0, logp, torch.zeros_like(logp))
    soft = p * (total[:, None] + h.double()[:, None] * (safe + ent[:, None]))
    d = -soft
    d.scatter_add_(1, t.long().clamp(0, v - 1)[:, None], g[:, None])
    if top:
        d.scatter_add_(1, ids.clamp(min=0), a.double())
    d *= inv
    d[empty] = 0
    d[bad] = math.nan
    # |parts| of an entry: what the relative errors of p and the fp32 roundings act on
    size = p * (total.abs()[:, None] + a.double().abs().sum(1)[:, None] + h.double().abs()[:, None] *
                (safe.abs() + ent.abs()[:, None] + 1))
    one = torch.zeros_like(size)
    one.scatter_add_(1, t.long().clamp(0, v - 1)[:, None], g.abs()[:, None])
    if top:
        one.scatter_add_(1, ids.clamp(min=0), a.double().abs())
    return d, size * inv, one * inv


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,v,top,pad,temperature", [(1, 1, 1, 0, 1.0), (3, 7, 2, 1, 1.0), (5, 1000, 8, 3, 0.7),
                                                     (40, 515, 64, 0, 1.3), (4, 32003, 20, 5, 1.0),
                                                     (900, 301, 0, 0, 1.0)])
def test_gradient_formula(m, v, top, pad, temperature, dtype):
    z, t = _logits(m * v, m, v, dtype, pad)
    if m > 3:
        z[0] = -math.inf
        z[1, :: 2] = -math.inf
        t[2] = -100
        t[3] = v + 5
    if m > 30:
        z[4, 1] = math.nan
    gen = torch.Generator().manual_seed(v)
    g, h = (torch.randn(m, generator=gen).to(DEV) for _ in range(2))
    a = torch.randn(m, top, generator=gen).to(DEV)
    leaf = z.detach().requires_grad_()
    r = w4.token_logprobs(leaf, t, top=top, temperature=temperature)
    outs = [r.logprobs, r.entropy] + ([r.top_logprobs] if top else [])
    (dz,) = torch.autograd.grad(outs, leaf, [g, h] + ([a] if top else []))
    ref, size, one = _gradient(z, t, top, temperature, g, h, a)
    # p's relative error is the absolute error of its logarithm (its exponent's rounding among it)
    tol = _tol(z, temperature) * 4 * size + 2.0**-24 * 8 * (size + one)
    tol = tol + (HALF_ULP[dtype] * (ref.abs() + tol) + TINY[dtype])
    assert dz.dtype == dtype
    bad = torch.isnan(ref)
    assert torch.equal(torch.isnan(dz), bad)
    d = torch.where(bad, torch.zeros_like(ref), (dz.double() - ref).abs())
    assert (d <= torch.where(bad, torch.ones_like(tol), tol)).all(), d.max()


@pytest.mark.gpu
def test_gradient_differences():
    """Central differences of the operator: third derivatives of every output are below 6 in
    magnitude here, fp32 outputs carry 1e-6."""
    m, v, top, eps = 4, 37, 3, 2.0**-6
    z, t = _logits(9, m, v, torch.float32, spread=1.0)
    z = z.contiguous()
    gen = torch.Generator().manual_seed(1)
    g, h = (torch.randn(m, generator=gen).to(DEV) for _ in range(2))
    a = torch.randn(m, top, generator=gen).to(DEV)
    leaf = z.clone().requires_grad_()
    r = w4.token_logprobs(leaf, t, top=top, temperature=0.8)
    (dz,) = torch.autograd.grad([r.logprobs, r.entropy, r.top_logprobs], leaf, [g, h, a])

    def f(x):
        s = w4.token_logprobs(x, t, top=top, temperature=0.8)
        same = (s.top_ids == r.top_ids).all(1)
        return ((s.logprobs * g).double() + (s.entropy * h).double() + (s.top_logprobs * a).double().sum(1)), same

    coef = (g.abs() + h.abs() * (1 + math.log(v)) + a.abs().sum(1)).double()
    for j in range(v):
        up, dn = z.clone(), z.clone()
        up[:, j] += eps
        dn[:, j] -= eps
        (fu, su), (fd, sd) = f(up), f(dn)
        ok = su & sd  # the alternatives are the same tokens on both sides
        tol = coef * (eps * eps * 6 / (6 * 0.8**3) + 1e-6 / eps)
        assert ((((fu - fd) / (2 * eps) - dz[:, j].double()).abs() <= tol) | ~ok).all(), j


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["logprobs", "entropy", "top_logprobs"])
def test_gradient_of_one_output(which):
    z, t = _logits(17, 6, 211, torch.float32)
    leaf = z.clone().requires_grad_()
    out = getattr(w4.token_logprobs(leaf, t, top=4), which)
    out.sum().backward()  # a broadcast gradient
    ref = z.double().requires_grad_()
    lp = torch.log_softmax(ref, 1)
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :4]
    want = {"logprobs": lp.gather(1, t[:, None]), "entropy": -(lp.exp() * lp).sum(1), "top_logprobs": lp.gather(1, ids)}
    want[which].sum().backward()
    assert (leaf.grad.double() - ref.grad).abs().max() < 2e-5  # coefficients of at most 4, p <= 1


@pytest.mark.gpu
def test_no_rows_and_stream():
    r = w4.token_logprobs(torch.empty(0, 50, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV), top=3)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 3)
    z, t = _logits(5, 3, 60000, torch.bfloat16)
    want = w4.token_logprobs(z, t, top=9)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        got = w4.token_logprobs(z, t, top=9)
    st.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("m,v", [(2, 128256), (64, 9000)])
def test_graph_replays(m, v):
    z, t = _logits(1, m, v, torch.bfloat16)
    z = z.contiguous()
    w4.token_logprobs(z, t, top=5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = w4.token_logprobs(z, t, top=5)
    for i in range(3):
        z.copy_(_logits(10 + i, m, v, torch.bfloat16)[0])
        want = w4.token_logprobs(z, t, top=5)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, r):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_more_rows_than_a_launch_holds():
    """2^24 + 3 rows of two logits: log p of the first is -log(1 + e^d) exactly, d = z1 - z0."""
    M = (1 << 24) + 3
    gen = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn(M, 2, device="cuda", generator=gen).requires_grad_()
    t = torch.randint(2, (M,), device="cuda", generator=gen)
    s = w4.token_logprobs(z, t, top=1)
    d = z.detach().double()
    d = (d[:, 0] - d[:, 1]) * (2 * t - 1)  # other minus target
    ref = -torch.nn.functional.softplus(d)
    # fp32: the difference (2^-24 of it), exp2, a sum of two and a logarithm, each some 2^-22
    assert (s.logprobs.double() - ref).abs().max() < 1e-5
    assert torch.equal(s.top_ids[:, 0], (z.detach()[:, 1] > z.detach()[:, 0]).long())
    s.logprobs.sum().backward()
    q = torch.sigmoid(d)  # the other's probability
    ref = torch.stack([torch.where(t == 0, q, -q), torch.where(t == 1, q, -q)], 1)
    assert (z.grad.double() - ref).abs().max() < 1e-5


def _plain_launches(monkeypatch):
    """The launches of the scores replaced by torch on the CPU: what is left is the autograd."""
    from gemv_int4_quantize_amd import scores

    def forward(z, t, top, temperature, ignore):
        lp = torch.log_softmax(z / temperature, 1)
        v, ids = lp.topk(top, 1)
        return lp.gather(1, t[:, None])[:, 0], -(lp.exp() * lp).sum(1), v, ids, torch.zeros(z.shape[0], 2)

    def grad(z, t, stats, ent, ids, top, g, h, a, temperature, ignore, out):
        out.copy_(torch.zeros_like(z) if g is None else
                  g[:, None] * (torch.nn.functional.one_hot(t, z.shape[1]) - torch.softmax(z / temperature, 1)) / temperature)

    monkeypatch.setattr(scores, "_forward", forward)
    monkeypatch.setattr(scores, "_grad", grad)


def test_second_derivatives_raise(monkeypatch):
    """The gradient is no function that autograd knows: a second derivative through it raises, and is
    not silently that of the loss's other terms alone."""
    _plain_launches(monkeypatch)
    t = torch.tensor([1, 2])
    for weight in (torch.ones(2), torch.ones(2, requires_grad=True)):
        z = torch.randn(2, 5, requires_grad=True)
        loss = (w4.token_logprobs(z, t).logprobs * weight).sum() + (z**3).sum()
        (g,) = torch.autograd.grad(loss, z, create_graph=True)
        with pytest.raises(RuntimeError, match="twice|once_differentiable"):
            g.square().sum().backward()
    # the first derivative is as it was, also with the graph kept
    z = torch.randn(2, 5, requires_grad=True)
    w4.token_logprobs(z, t).logprobs.sum().backward(retain_graph=True)
    one = torch.nn.functional.one_hot(t, 5)
    assert torch.allclose(z.grad, one - torch.softmax(z.detach(), 1))


def test_forward_mode_raises(monkeypatch):
    """No tangent is computed: a dual tensor raises, and its tangent is not silently dropped."""
    import torch.autograd.forward_ad as fwd

    _plain_launches(monkeypatch)
    t = torch.tensor([1, 2])
    with fwd.dual_level():
        for grad in (False, True):
            z = fwd.make_dual(torch.randn(2, 5, requires_grad=grad), torch.randn(2, 5))
            with pytest.raises(RuntimeError, match="forward"):
                w4.token_logprobs(z, t)
            with pytest.raises(RuntimeError, match="forward"), torch.no_grad():
                w4.token_logprobs(z.t().contiguous().t(), t)
        assert w4.token_logprobs(torch.randn(2, 5), t).logprobs.shape == (2,)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,v", [(500, 17003), (250, 33001), (9, 70001), (1, 17003), (1100, 5003)])
def test_every_column_counts_once(m, v, dtype):
    """Rows of two logits, all else masked: one at a column of its own, which goes over the whole row
    (over the edges of every 64 columns where that is too much), one at the first or the last.  Each
    has probability 1/2: a logit lost or counted twice at a part's or a run's edge would show as
    log p = 0 or -log 3, and a column without its gradient as a value other than +-1/2."""
    cols = torch.arange(1, v - 1, device=DEV)
    if m < 100:
        cols = cols[(cols % 64 < 2) | (cols % 64 > 62)]
        cols = cols[:: max(1, len(cols) // (m * 60)) | 1]
    half = torch.full((m,), -math.log(2.0), device=DEV)
    rows = torch.arange(m, device=DEV)
    for at in range(0, len(cols), m):
        j = cols[at:at + m]
        j = torch.cat([j, cols[:m - len(j)]])
        other = torch.where(rows % 2 == 0, 0, v - 1)
        z = torch.full((m, v), -math.inf, dtype=dtype, device=DEV)
        z[rows, j] = 4.0
        z[rows, other] = 4.0
        r = w4.token_logprobs(z, j, top=2)
        # one logarithm of 2 (2^-24 of it and of its half ulp)
        assert (r.logprobs - half).abs().max() <= 2.0**-22 and (r.entropy + half).abs().max() <= 2.0**-22, at
        assert torch.equal(r.top_ids, torch.stack([torch.minimum(j, other), torch.maximum(j, other)], 1)), at
        dz = w4.token_logprobs_grad(z, j, r.stats, r.entropy, r.top_ids, torch.ones(m, device=DEV))
        want = torch.zeros_like(dz)
        want[rows, j], want[rows, other] = 0.5, -0.5
        assert ((dz - want).abs() <= 2.0**-20).all(), at


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 200, 1100])
def test_equal_logits_sum_to_their_number(m):
    """A row of equal logits at a number of columns that fp32 counts exactly: log p = -log V."""
    for v in (4096, 65536, 131072, 17003, 40001):
        if m * v > 1 << 27:
            continue
        z = torch.full((m, v), -3.0, device=DEV)
        r = w4.token_logprobs(z, torch.full((m,), v - 1, device=DEV))
        # terms of 1 and sums of whole numbers are exact: one logarithm and its rounding are left
        assert (r.logprobs.double() + math.log(v)).abs().max() <= 2.0**-20, v
        assert (r.entropy.double() - math.log(v)).abs().max() <= 2.0**-20, v
