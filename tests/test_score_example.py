"""examples/score_tokens.py: the operators run together, against 64-bit arithmetic on the CPU."""

import importlib.util
import os

import pytest
import torch

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "score_tokens.py")


def _example():
    spec = importlib.util.spec_from_file_location("score_tokens", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_imports():
    m = _example()
    assert callable(m.build) and callable(m.train)


@pytest.mark.gpu
def test_scores_and_decoding():
    m = _example()
    head, _, embed, x, t = m.build(33, 192, 1003)
    s = m.score_prompt(head, x, t)
    # of the head's own bf16 logits: only fp32 sums of 1003 terms separate the two
    z = head(x).double().cpu()
    ref = torch.log_softmax(z, 1)
    torch.testing.assert_close(s.logprobs.double().cpu(), ref.gather(1, t.cpu()[:, None])[:, 0], rtol=0, atol=2e-5)
    assert (ref.gather(1, s.top_ids.cpu()) >= ref.topk(5).values - 1e-12).all()
    # the logits: codes * scales of both sides, exact sums, one fp32 and one bf16 rounding (2^-8)
    q = m.w4.quantize_int8(x)
    full = (q.codes[:, :192].double().cpu() * q.scales.double().cpu()[:, None]) @ \
           (head.w.codes[:, :192].double().cpu() * head.w.scales.double().cpu()[:, None]).T
    assert ((z - full).abs() <= full.abs() * 2.0 ** -8 + 1e-30).all()
    # the decoded tokens follow one another
    state = x[-1:]
    for tok, lp in m.decode(head, embed, state, 4):
        row = torch.log_softmax(head(state).double().cpu(), 1)[0]
        assert row[tok] == row.max() and abs(float(row[tok]) - lp) < 2e-5
        state = embed[tok:tok + 1]


@pytest.mark.gpu
def test_training_step_gradient():
    """The gradient at the hidden states and at the adapter against the formula in 64 bits."""
    m = _example()
    M, H, V, h = 24, 128, 515, 0.01
    head, adapter, _, x, t = m.build(M, H, V)
    xg = x.clone().requires_grad_()
    a0 = adapter.a.detach().clone()
    y = head(xg)
    s = m.w4.token_logprobs(y, t)
    (-(s.logprobs.mean() + h * s.entropy.mean())).backward()
    z = y.detach().double().cpu()
    lp = torch.log_softmax(z, 1)
    p = lp.exp()
    ent = -(p * lp).sum(1, keepdim=True)
    one = torch.nn.functional.one_hot(t.cpu(), V).double()
    dz = -((one - p) - h * p * (lp + ent)) / M
    w = (head.w.codes[:, :H].float() * head.w.scales[:, None]).bfloat16().double().cpu()
    ref = dz @ w
    # dz and dX each rounded to bf16 (2^-8 of a term, of the result), fp32 sums below both
    bound = (dz.abs() @ w.abs()) * (2.0 ** -8 + 2.0 ** -14) + ref.abs() * 2.0 ** -8 + 1e-12
    assert ((xg.grad.double().cpu() - ref).abs() <= bound).all()
    # one training step: at B = 0 the adapter's inner gradient is (x A)^T dX, A's is 0; fp32 products of 24 and 128 terms
    losses = m.train(head, adapter, x, t, 1)
    assert abs(losses[0] + float(lp.gather(1, t.cpu()[:, None]).mean() + h * ent.mean())) < 2e-5
    xa, dx = x.double().cpu() @ a0.double().cpu(), xg.grad.double().cpu()
    mag = (x.double().cpu().abs() @ a0.double().cpu().abs()).T @ dx.abs()
    assert ((adapter.b.grad.double().cpu() - xa.T @ dx).abs() <= mag * 2.0 ** -16).all()
    assert (adapter.a.grad == 0).all()
