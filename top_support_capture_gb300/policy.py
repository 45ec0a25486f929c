"""A policy's whole vocabulary: log-probabilities of given tokens with the entropy and the top alternatives, their
gradient, and the clipped policy loss with its gradient.

Like the rest of the binding this only checks and marshals arguments (include/sfc.h has the formulas). The functions ending
in ``_backward`` / ``_and_grad`` take no part in autograd: a training step that is captured into a CUDA graph uses those.
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd import forward_ad

from . import FLAG_TEST_STALL, MAX_GIVEN, MAX_TOP, SFC_OK, SfcError, _dtype_code, _enter, _expect, _ptr, load_library
from .training import _check_grad, _raise, _rows_args, check_derivatives, check_rows


class TokenLogprobs(NamedTuple):
    logprobs: "object"  # float32, the tokens' shape, or None (no tokens)
    entropy: "object"  # float32 [B]
    top_ids: "object"  # int32 [B, top], or None
    top_logprobs: "object"  # float32 [B, top], or None
    row_status: "object"  # int32 [B]
    row_stats: "object" = None  # float32 [B, 4] for token_logprobs_backward, or None


class PolicyGradOutput(NamedTuple):
    loss: "object"  # float32 [B]
    logprobs: "object"  # float32 [B]
    entropy: "object"  # float32 [B]
    grad_logits: "object"  # [B, V], the logits' dtype
    row_status: "object"  # int32 [B]


def check_tokens(logits, tokens, most=MAX_GIVEN):
    """int32 tokens [B] or [B, M] beside [B, V] logits, or None; returns M."""
    if tokens is None:
        return 0
    shape = tokens.shape
    if len(shape) not in (1, 2) or shape[0] != logits.shape[0]:
        raise SfcError("tokens must be [B] or [B, M]")
    M = 1 if len(shape) == 1 else shape[1]
    if M < 1 or M > most:
        raise SfcError(f"tokens must be 1 to {most} a row, got {M}")
    _expect("tokens", tokens, logits.device, torch.int32)
    return M


def _forward(logits, stride, temperature, tokens, M, top, stream, keep_stats):
    dev, (B, V) = logits.device, logits.shape
    stream, context = _enter(dev, stream, logits, temperature, tokens)
    logprobs = ids = lps = stats = to_tokens = to_logprobs = to_ids = to_lps = to_stats = None
    with context:
        if M:
            logprobs = torch.empty(tokens.shape, dtype=torch.float32, device=dev)
            to_tokens, to_logprobs = tokens.data_ptr(), logprobs.data_ptr()
        entropy = torch.empty(B, dtype=torch.float32, device=dev)
        if top:
            ids, lps = torch.empty((B, top), dtype=torch.int32, device=dev), torch.empty((B, top), dtype=torch.float32, device=dev)
            to_ids, to_lps = ids.data_ptr(), lps.data_ptr()
        if keep_stats:
            stats = torch.empty((B, 4), dtype=torch.float32, device=dev)
            to_stats = stats.data_ptr()
        status = torch.empty(B, dtype=torch.int32, device=dev)
        rc = load_library().sfc_token_logprobs(logits.data_ptr(), _dtype_code(logits), B, V, stride, temperature.data_ptr(), to_tokens, M, top,
                                               to_logprobs, entropy.data_ptr(), to_ids, to_lps, to_stats, status.data_ptr(), stream)
    if rc != SFC_OK:
        _raise("sfc_token_logprobs", rc)
    return TokenLogprobs(logprobs, entropy, ids, lps, status, stats)


class _TokenLogprobs(torch.autograd.Function):
    """Makes the float outputs of a call that has been made already functions of its logits. (What goes through `apply` costs
    a few microseconds for each tensor: the whole numbers do not.)"""

    @staticmethod
    def forward(ctx, logits, temperature, tokens, out):
        ctx.save_for_backward(logits, temperature, tokens, out.row_stats, out.top_ids)
        ctx.has = out.logprobs is not None, out.top_logprobs is not None
        ctx.set_materialize_grads(False)  # none is made for what takes no part in a loss
        return tuple(t for t in (out.entropy, out.logprobs, out.top_logprobs) if t is not None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_entropy, *grads):
        grads = iter(grads)
        grad_logprobs, grad_top = (next(grads) if has else None for has in ctx.has)
        if grad_logprobs is None and grad_top is None and grad_entropy is None:
            return (None,) * 4
        logits, temperature, tokens, stats, top_ids = ctx.saved_tensors
        row = check_rows("logits", logits)  # (hooks on saved tensors may have laid them out anew)
        dev, (B, V) = logits.device, logits.shape
        stream, context = _enter(dev, None)  # autograd runs a backward on its forward's stream
        with context:
            if grad_top is not None:  # the alternatives are tokens like the others
                if grad_logprobs is None:
                    tokens, grad_logprobs = top_ids, grad_top
                else:
                    tokens = torch.cat((tokens.view(B, -1), top_ids), 1)
                    grad_logprobs = torch.cat((grad_logprobs.reshape(B, -1), grad_top), 1)
            elif grad_logprobs is None:
                tokens = None
            if grad_logprobs is not None and not (grad_logprobs.dtype is torch.float32 and grad_logprobs.is_contiguous()):
                grad_logprobs = grad_logprobs.to(torch.float32).contiguous()
            if grad_entropy is not None and not (grad_entropy.dtype is torch.float32 and grad_entropy.is_contiguous()):
                grad_entropy = grad_entropy.to(torch.float32).contiguous()
            grad = torch.empty((B, V), dtype=logits.dtype, device=dev)
            rc = load_library().sfc_token_logprobs_backward(
                *_rows_args(logits, row, temperature), _ptr(tokens), 0 if tokens is None else tokens.numel() // B, stats.data_ptr(),
                _ptr(grad_logprobs), _ptr(grad_entropy), grad.data_ptr(), V, stream)
        if rc != SFC_OK:
            _raise("sfc_token_logprobs_backward", rc)
        return grad, None, None, None


def token_logprobs(logits, temperature, tokens=None, top: int = 0, keep_stats: bool = False, stream=None) -> TokenLogprobs:
    """Log-probabilities over the whole vocabulary of ``logits`` [B, V] (bf16/f32 CUDA) at the per-row ``temperature``: those
    of the given ``tokens`` ([B] or [B, M] int32, -1 for none), each row's entropy, and its ``top`` most likely tokens
    (ties to the lowest id). Differentiable in ``logits`` (reverse mode), and in nothing else: a ``temperature`` that requires a
    gradient is refused. ``keep_stats`` gives the ``row_stats`` that ``token_logprobs_backward`` takes. See include/sfc.h."""
    row = check_rows("logits", logits)
    M, top = check_tokens(logits, tokens), int(top)
    if top < 0 or top > MAX_TOP:
        raise SfcError(f"top must be 0 to {MAX_TOP}, got {top}")
    _expect("temperature", temperature, logits.device, torch.float32, numel=logits.shape[0])
    if temperature.requires_grad or getattr(forward_ad, "_current_level", 0) >= 0:
        check_derivatives(logits, temperature=temperature)
    if torch.is_grad_enabled() and logits.requires_grad:
        if keep_stats:
            raise SfcError("keep_stats is for calls outside autograd: detach the logits")
        _, context = _enter(logits.device, stream, logits, temperature, tokens)
        with context:
            out = _forward(logits, row, temperature, tokens, M, top, None, True)
            floats = iter(_TokenLogprobs.apply(logits, temperature, tokens, out))
            entropy = next(floats)
            return TokenLogprobs(next(floats) if M else None, entropy, out.top_ids, next(floats) if top else None, out.row_status)
    return _forward(logits, row, temperature, tokens, M, top, stream, keep_stats)


def token_logprobs_backward(logits, temperature, tokens, row_stats, grad_logprobs=None, grad_entropy=None, grad=None, stream=None):
    """The gradient of ``token_logprobs`` with respect to ``logits`` [B, V], from the ``row_stats`` [B, 4] that the call gave
    for the same logits and temperatures and the upstream gradients ``grad_logprobs`` (f32, the tokens' shape) and
    ``grad_entropy`` [B] f32, either of which may be None: a dense [B, V] tensor of the logits' dtype (written into ``grad``
    when that is given). Up to 128 tokens a row: for gradients of top alternatives their ids are given as tokens."""
    row = check_rows("logits", logits)
    dev, B = logits.device, logits.shape[0]
    M = check_tokens(logits, tokens, MAX_GIVEN + MAX_TOP)
    _expect("temperature", temperature, dev, torch.float32, numel=B)
    if row_stats is None:
        raise SfcError("row_stats is required (token_logprobs with keep_stats)")
    _expect("row_stats", row_stats, dev, torch.float32, shape=(B, 4))
    if grad_logprobs is not None:
        if tokens is None:
            raise SfcError("grad_logprobs needs tokens")
        _expect("grad_logprobs", grad_logprobs, dev, torch.float32, shape=tokens.shape)
    if grad_entropy is not None:
        _expect("grad_entropy", grad_entropy, dev, torch.float32, numel=B)
    grad_row = logits.shape[1] if grad is None else _check_grad(grad, logits)
    stream, context = _enter(dev, stream, logits, temperature, tokens, row_stats, grad_logprobs, grad_entropy, grad)
    with context:
        if grad is None:
            grad = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        rc = load_library().sfc_token_logprobs_backward(*_rows_args(logits, row, temperature), _ptr(tokens), M, row_stats.data_ptr(),
                                                        _ptr(grad_logprobs), _ptr(grad_entropy), grad.data_ptr(), grad_row, stream)
    if rc != SFC_OK:
        _raise("sfc_token_logprobs_backward", rc)
    return grad


def policy_loss_and_grad(logits, temperature, tokens, advantages, grad_loss, old_logprobs=None, clip_low: float = 0.2,
                         clip_high: float = 0.2, entropy_weight: float = 0.0, grad=None, stream=None,
                         test_stall: bool = False) -> PolicyGradOutput:
    """The clipped policy loss of the sampled ``tokens`` [B] int32 (-1: padding) under ``logits`` [B, V] and its gradient in
    one call, for a known upstream gradient ``grad_loss`` [B] f32 (a mean over the batch: 1 / B each): the logits are read
    once. ``advantages`` [B] f32; ``old_logprobs`` [B] f32 are the sampling policy's, as ``token_logprobs`` gives them at the
    same temperature; without them the loss is the weighted cross-entropy. ``grad`` may give the [B, V] tensor to write (not
    the logits themselves). Outside autograd. See include/sfc.h."""
    row = check_rows("logits", logits)
    dev, f32, (B, V) = logits.device, torch.float32, logits.shape
    _expect("temperature", temperature, dev, f32, numel=B)
    _expect("tokens", tokens, dev, torch.int32, shape=(B,))
    _expect("advantages", advantages, dev, f32, numel=B)
    _expect("grad_loss", grad_loss, dev, f32, numel=B)
    if old_logprobs is not None:
        _expect("old_logprobs", old_logprobs, dev, f32, numel=B)
    grad_row = V if grad is None else _check_grad(grad, logits)
    stream, context = _enter(dev, stream, logits, temperature, tokens, advantages, grad_loss, old_logprobs, grad)
    with context:
        loss, logprobs = torch.empty(B, dtype=f32, device=dev), torch.empty(B, dtype=f32, device=dev)
        entropy, status = torch.empty(B, dtype=f32, device=dev), torch.empty(B, dtype=torch.int32, device=dev)
        if grad is None:
            grad = torch.empty((B, V), dtype=logits.dtype, device=dev)
        rc = load_library().sfc_policy_forward_backward(
            logits.data_ptr(), _dtype_code(logits), B, V, row, temperature.data_ptr(), tokens.data_ptr(),
            None if old_logprobs is None else old_logprobs.data_ptr(), advantages.data_ptr(), clip_low, clip_high, entropy_weight,
            FLAG_TEST_STALL if test_stall else 0, grad_loss.data_ptr(), loss.data_ptr(), logprobs.data_ptr(), entropy.data_ptr(),
            status.data_ptr(), grad.data_ptr(), grad_row, stream)
    if rc != SFC_OK:
        _raise("sfc_policy_forward_backward", rc)
    return PolicyGradOutput(loss, logprobs, entropy, grad, status)
