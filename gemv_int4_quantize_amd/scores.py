"""Log probabilities of given tokens with entropy and top alternatives, differentiable.

``token_logprobs`` reads the logits once and returns, for each row, the log probability of its
target, the entropy of its distribution and its k most likely tokens; the backward pass
writes the gradient with respect to the logits in one more pass.  Neither forms the
log-softmax.  The arithmetic runs in the library's gfx950 kernels (include/w8a8.h).
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._lib import check, lib
from .int8 import _row_stride, float_rows, on_device
from .ops import _WDT, _stream


class TokenLogprobs(NamedTuple):
    """Scores of M rows: fp32 [M], fp32 [M], fp32 [M][k], int64 [M][k], and fp32 [M][2]: the row's
    largest logit and the logarithm of the sum above it, which ``token_logprobs_grad`` takes."""

    logprobs: torch.Tensor
    entropy: torch.Tensor
    top_logprobs: torch.Tensor
    top_ids: torch.Tensor
    stats: torch.Tensor


def _forward(z, t, top, temperature, ignore):
    M, V = z.shape
    lp = torch.empty(M, dtype=torch.float32, device=z.device)
    ent = torch.empty(M, dtype=torch.float32, device=z.device)
    stats = torch.empty((M, 2), dtype=torch.float32, device=z.device)
    top_lp = torch.empty((M, top), dtype=torch.float32, device=z.device)
    ids = torch.empty((M, top), dtype=torch.int64, device=z.device)
    size = ctypes.c_size_t(0)
    with on_device(z, t):
        L = lib()
        check(L.tok_workspace_bytes(M, V, top, ctypes.byref(size)))
        ws = torch.empty(size.value, dtype=torch.uint8, device=z.device) if size.value else None
        check(L.tok_logprobs(z.data_ptr(), _WDT[z.dtype], M, V, _row_stride(z), t.data_ptr(), ignore, temperature, top,
                             lp.data_ptr(), ent.data_ptr(), stats.data_ptr(), top_lp.data_ptr() if top else None,
                             ids.data_ptr() if top else None, ws.data_ptr() if ws is not None else None, size.value,
                             _stream(z.device)))
    return lp, ent, top_lp, ids, stats


def token_logprobs_grad(logits: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor, entropy: torch.Tensor,
                        top_ids: torch.Tensor, grad_logprobs=None, grad_entropy=None, grad_top=None,
                        temperature: float = 1.0, ignore_index: int = -100,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient with respect to the logits of the scores whose gradients are given (None: zero).
    `out` may be the logits themselves, which it then replaces."""
    z = logits
    M, V = z.shape
    top = top_ids.shape[1]
    if out is None:
        out = torch.empty((M, V), dtype=z.dtype, device=z.device)
    elif out.shape != z.shape or out.dtype != z.dtype or (V > 1 and out.stride(1) != 1):
        raise ValueError("out must have the logits' shape and dtype and contiguous rows")
    g, h, a = (None if x is None else x.to(torch.float32).contiguous()
               for x in (grad_logprobs, grad_entropy, grad_top if top else None))
    with on_device(z, targets, stats, entropy, top_ids, g, h, a, out):
        check(lib().tok_logprobs_grad(
            z.data_ptr(), _WDT[z.dtype], M, V, _row_stride(z), targets.data_ptr(), ignore_index, temperature, top,
            stats.data_ptr(), entropy.data_ptr(), top_ids.data_ptr() if top else None,
            *(None if x is None else x.data_ptr() for x in (g, h, a)), out.data_ptr(), _row_stride(out),
            _stream(z.device)))
    return out


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
        dz = token_logprobs_grad(z, t, stats, ent, ids, g, h, a, ctx.temperature, ctx.ignore)
        return dz, None, None, None, None


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
    float results are differentiable with respect to the logits."""
    z = float_rows(logits, "logits")
    if targets.shape != (z.shape[0],) or targets.dtype not in (torch.int64, torch.int32):
        raise ValueError(f"targets must be an int64 or int32 vector of length {z.shape[0]}")
    t = targets.to(torch.int64).contiguous()
    if torch.is_grad_enabled() and z.requires_grad:
        return TokenLogprobs(*_TokenLogprobs.apply(z, t, int(top), float(temperature), int(ignore_index)))
    return TokenLogprobs(*_forward(z.detach(), t, int(top), float(temperature), int(ignore_index)))
