"""Log probabilities of given tokens with entropy and top alternatives, differentiable.

``token_logprobs`` reads the logits once and returns, for each row, the log probability of its
target, the entropy of its distribution and its k most likely tokens; the backward pass
writes the gradient with respect to the logits in one more pass.  Neither forms the
log-softmax.  The arithmetic runs in the library's gfx950 kernels (include/w8a8.h).
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch
from torch.autograd.forward_ad import unpack_dual

from ._lib import check, lib
from .int8 import _row_stride, check_device, float_rows, on_device, once, space
from .ops import _WDT, _stream


class TokenLogprobs(NamedTuple):
    """Scores of M rows: fp32 [M], fp32 [M], fp32 [M][k], int64 [M][k], and fp32 [M][2]: the row's
    largest logit and the logarithm of the sum above it, which ``token_logprobs_grad`` takes."""

    logprobs: torch.Tensor
    entropy: torch.Tensor
    top_logprobs: torch.Tensor
    top_ids: torch.Tensor
    stats: torch.Tensor


@functools.lru_cache(maxsize=4096)
def _bytes(M: int, V: int, top: int) -> int:
    """Workspace of a call, which depends on its sizes alone."""
    size = ctypes.c_size_t(0)
    check(lib().tok_workspace_bytes(M, V, top, ctypes.byref(size)))
    return size.value


def _forward(z, t, top, temperature, ignore):
    M, V = z.shape
    lp = torch.empty(M, dtype=torch.float32, device=z.device)
    ent = torch.empty(M, dtype=torch.float32, device=z.device)
    stats = torch.empty((M, 2), dtype=torch.float32, device=z.device)
    top_lp = torch.empty((M, top), dtype=torch.float32, device=z.device)
    ids = torch.empty((M, top), dtype=torch.int64, device=z.device)
    with on_device(check_device(z, t)):
        size = _bytes(M, V, top)
        ws = space(size, z.device)
        status = lib().tok_logprobs(
            z.data_ptr(), _WDT[z.dtype], M, V, _row_stride(z), t.data_ptr(), ignore, temperature, top, lp.data_ptr(),
            ent.data_ptr(), stats.data_ptr(), top_lp.data_ptr() if top else None, ids.data_ptr() if top else None,
            ws.data_ptr() if ws is not None else None, size, _stream(z.device))
    check(status)
    return lp, ent, top_lp, ids, stats


def token_logprobs_grad(logits: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor, entropy: torch.Tensor,
                        top_ids: torch.Tensor, grad_logprobs=None, grad_entropy=None, grad_top=None,
                        temperature: float = 1.0, ignore_index: int = -100,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient with respect to the logits of the scores whose gradients are given (None: zero).
    `out` may be the logits themselves, which it then replaces."""
    z = float_rows(logits, "logits")
    M, V = z.shape
    t = _targets(targets, M)
    top = top_ids.shape[1] if top_ids.dim() == 2 else -1
    for x, what, dtype, shape in ((stats, "stats", torch.float32, (M, 2)), (entropy, "entropy", torch.float32, (M,)),
                                  (top_ids, "top_ids", torch.int64, (M, top))):
        if x.dtype != dtype or x.shape != shape or not x.is_contiguous():
            raise ValueError(f"{what} must be the contiguous {dtype} tensor of shape {shape} that token_logprobs gave")
    for x, what, shape in ((grad_logprobs, "grad_logprobs", (M,)), (grad_entropy, "grad_entropy", (M,)),
                           (grad_top, "grad_top", (M, top))):
        if x is not None and x.shape != shape:
            raise ValueError(f"{what} must have shape {shape}")
    if out is None:
        out = torch.empty((M, V), dtype=z.dtype, device=z.device)
    elif out.shape != z.shape or out.dtype != z.dtype or (V > 1 and out.stride(1) != 1):
        raise ValueError("out must have the logits' shape and dtype and contiguous rows")
    g, h, a = (_plain_grad(x) for x in (grad_logprobs, grad_entropy, grad_top if top else None))
    with on_device(check_device(z, t, stats, entropy, top_ids, g, h, a, out)):
        _grad(z, t, stats, entropy, top_ids, top, g, h, a, temperature, ignore_index, out)
    return out


def _targets(targets: torch.Tensor, M: int) -> torch.Tensor:
    if targets.shape != (M,) or targets.dtype not in (torch.int64, torch.int32):
        raise ValueError(f"targets must be an int64 or int32 vector of length {M}")
    return targets.to(torch.int64).contiguous()


def _plain_grad(x):
    """A gradient as the library takes it (None: zero): fp32, contiguous."""
    if x is None or (x.dtype is torch.float32 and x.is_contiguous()):
        return x
    return x.to(torch.float32).contiguous()


def _grad(z, t, stats, ent, ids, top, g, h, a, temperature, ignore, out):
    M, V = z.shape
    check(lib().tok_logprobs_grad(
        z.data_ptr(), _WDT[z.dtype], M, V, _row_stride(z), t.data_ptr(), ignore, temperature, top, stats.data_ptr(),
        ent.data_ptr(), ids.data_ptr() if top else None, None if g is None else g.data_ptr(),
        None if h is None else h.data_ptr(), None if a is None else a.data_ptr(), out.data_ptr(), _row_stride(out),
        _stream(z.device)))


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, t, top, temperature, ignore):
        lp, ent, top_lp, ids, stats = _forward(z, t, top, temperature, ignore)
        ctx.save_for_backward(z, t, stats, ent, ids)
        ctx.temperature, ctx.ignore = temperature, ignore
        ctx.mark_non_differentiable(ids, stats)
        ctx.set_materialize_grads(False)
        return lp, ent, top_lp, ids, stats

    @staticmethod
    def backward(ctx, g, h, a, *_):
        if g is None and h is None and a is None:
            return None, None, None, None, None
        z, t, stats, ent, ids = ctx.saved_tensors
        # the engine has made the node's device current; its thread is cold, so little is done here
        dz = torch.empty(z.shape, dtype=z.dtype, device=z.device)
        top = ids.shape[1]
        _grad(z, t, stats, ent, ids, top, _plain_grad(g), _plain_grad(h), _plain_grad(a) if top else None,
              ctx.temperature, ctx.ignore, dz)
        return once(dz, "token_logprobs", z, g, h, a), None, None, None, None


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, top: int = 0, temperature: float = 1.0,
                   ignore_index: int = -100) -> TokenLogprobs:
    """Scores of one target token per row of logits [M][V] (float32, float16 or bfloat16; rows may
    be strided) under softmax(logits / temperature):

    * ``logprobs`` [M]: the target's log probability; 0 where the target is ``ignore_index``, NaN
      where it is outside the vocabulary otherwise;
    * ``entropy`` [M], in nats;
    * ``top_logprobs`` and ``top_ids`` [M][top]: the most likely tokens in order, ties to the lowest
      id (top <= 64).

    A logit of -inf is a masked token (probability 0).  A row that is masked throughout has log
    probabilities -inf, entropy 0 and no gradient; a row with a NaN or +inf scores NaN.  The three
    float results are differentiable with respect to the logits, once and in reverse
    mode: a second derivative and a tangent raise."""
    if unpack_dual(logits).tangent is not None:
        raise RuntimeError("token_logprobs has no derivative in forward mode")
    z = float_rows(logits, "logits")
    t = _targets(targets, z.shape[0])
    if torch.is_grad_enabled() and z.requires_grad:
        return TokenLogprobs(*_TokenLogprobs.apply(z, t, int(top), float(temperature), int(ignore_index)))
    return TokenLogprobs(*_forward(z.detach(), t, int(top), float(temperature), int(ignore_index)))
