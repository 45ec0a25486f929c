"""Training against captured supports: distillation from a teacher's top logits, and the replay's gradient.

Like the rest of the binding this only checks and marshals arguments (include/sfc.h has the formulas). The
functions ending in ``_backward`` / ``_and_grad`` take no part in autograd: a training step that is captured
into a CUDA graph uses those. (Autograd's own bookkeeping is not made for a captured backward pass while an
eager graph over the same leaves is alive.)
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd import forward_ad

from . import (FLAG_NORMALISE_TEACHER, FLAG_TEST_STALL, MAX_PACKED_WIDTH, SFC_OK, ReplayOutput, SfcError, _dtype_code, _enter, _expect, _ptr,
               load_library, replay_logprob, strerror)


class DistillOutput(NamedTuple):
    loss: "object"  # float32 [B]
    row_status: "object"  # int32 [B]


class DistillGradOutput(NamedTuple):
    loss: "object"  # float32 [B]
    grad_logits: "object"  # [B, V], the logits' dtype
    row_status: "object"  # int32 [B]


def check_rows(name, t):
    """[B, V] rows of a CUDA tensor, each contiguous; returns the row stride."""
    if not t.is_cuda:
        raise SfcError(f"{name} must be a CUDA tensor, got {t.device}")
    return check_row_layout(name, t)


def check_row_layout(name, t):
    """A floating [B, V] tensor whose rows are contiguous and do not overlap; returns the row stride."""
    if t.dim() != 2 or t.numel() < 1:
        raise SfcError(f"{name} must be a non-empty [B, V] tensor")
    _dtype_code(t)
    (B, V), (row, one) = t.shape, t.stride()
    if one != 1 and V > 1:
        raise SfcError(f"{name} rows must be contiguous")
    if row < V:
        if B > 1:
            raise SfcError(f"{name} rows must not overlap (an expanded tensor: make it contiguous)")
        row = V
    return row


def check_packed(logits, temperature, ids, lengths, values=None, values_name="teacher_values", ids_name="teacher_ids"):
    """The packed per-row arrays beside [B, V] logits, as the kernels assume them; returns (device, B, W)."""
    dev, B, shape = logits.device, logits.shape[0], ids.shape
    if len(shape) != 2 or shape[0] != B:
        raise SfcError(f"{ids_name} must be [B, W]")
    W = shape[1]
    if W < 1 or W > MAX_PACKED_WIDTH:
        raise SfcError(f"{ids_name} must be 1 to {MAX_PACKED_WIDTH} wide, got {W}")
    _expect(ids_name, ids, dev, torch.int32)
    _expect("temperature", temperature, dev, torch.float32, numel=B)
    _expect("lengths", lengths, dev, torch.int32, numel=B)
    if values is not None:
        _expect(values_name, values, dev, torch.float32, shape)
    return dev, B, W


def check_derivatives(logits, **constants):
    """Refuses derivatives that the calls here do not give, which would be lost without a word: forward-mode, and gradients
    of anything but the logits."""
    if getattr(forward_ad, "_current_level", 0) >= 0:  # (inside a dual level)
        for name, t in (("logits", logits), *constants.items()):
            if forward_ad.unpack_dual(t).tangent is not None:
                raise SfcError(f"{name} is a forward-mode dual tensor: there is no forward-mode derivative")
    if torch.is_grad_enabled():
        for name, t in constants.items():
            if t.requires_grad:
                raise SfcError(f"{name} requires a gradient, which is given for the logits only: detach it")


def _raise(name, rc):
    raise SfcError(f"{name}: {strerror(rc)} ({rc})")


def _check_grad(grad, logits):
    if grad.device != logits.device or grad.dtype != logits.dtype or grad.shape != logits.shape:
        raise SfcError("grad must have the logits' device, dtype and shape")
    return check_row_layout("grad", grad)


def _rows_args(logits, stride, temperature):
    B, V = logits.shape
    return logits.data_ptr(), _dtype_code(logits), B, V, stride, temperature.data_ptr()


def _teacher_args(ids, values, lengths, normalise, flags=0):
    return (ids.data_ptr(), values.data_ptr(), lengths.data_ptr(), ids.shape[1],
            flags | FLAG_NORMALISE_TEACHER if normalise else flags)


def _distill_forward(logits, stride, temperature, ids, values, lengths, normalise, stream, keep_stats):
    dev, B = logits.device, logits.shape[0]
    stream, context = _enter(dev, stream, logits, temperature, ids, values, lengths)
    with context:
        loss = torch.empty(B, dtype=torch.float32, device=dev)
        stats = torch.empty((B, 4), dtype=torch.float32, device=dev) if keep_stats else None
        status = torch.empty(B, dtype=torch.int32, device=dev)
        rc = load_library().sfc_distill_forward(*_rows_args(logits, stride, temperature), *_teacher_args(ids, values, lengths, normalise),
                                                loss.data_ptr(), _ptr(stats), status.data_ptr(), stream)
    if rc != SFC_OK:
        _raise("sfc_distill_forward", rc)
    return loss, stats, status


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, stride, temperature, ids, values, lengths, normalise):
        loss, stats, status = _distill_forward(logits, stride, temperature, ids, values, lengths, normalise, None, True)
        ctx.save_for_backward(logits, temperature, ids, values, lengths, stats)
        ctx.normalise, ctx.stride = normalise, stride
        ctx.set_materialize_grads(False)  # none is made for the status
        ctx.mark_non_differentiable(status)
        return loss, status

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, _):
        if grad_loss is None:
            return (None,) * 7
        logits, temperature, ids, values, lengths, stats = ctx.saved_tensors
        dev = logits.device
        stream, context = _enter(dev, None)  # autograd runs a backward on its forward's stream
        with context:
            grad_loss = grad_loss.to(torch.float32).contiguous()
            grad = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
            rc = load_library().sfc_distill_backward(*_rows_args(logits, ctx.stride, temperature),
                                                     *_teacher_args(ids, values, lengths, ctx.normalise), stats.data_ptr(),
                                                     grad_loss.data_ptr(), grad.data_ptr(), logits.shape[1], stream)
        if rc != SFC_OK:
            _raise("sfc_distill_backward", rc)
        return grad, None, None, None, None, None, None


def distill_loss(logits, temperature, teacher_ids, teacher_values, lengths, normalise: bool = False,
                 stream=None) -> DistillOutput:
    """Per-row distillation losses of a student's ``logits`` [B, V] (bf16/f32 CUDA) against packed teachers:
    ``teacher_ids`` [B, W] int32 with ``teacher_values`` [B, W] f32, log-probabilities (a capture's
    ``support_ids`` and ``support_logprobs``) or, with ``normalise``, raw top logits; ``lengths`` [B] int32 (0:
    the row has no teacher). Differentiable in ``logits`` (reverse mode), and in nothing else: a ``temperature`` or
    ``teacher_values`` that requires a gradient is refused. See include/sfc.h."""
    row = check_rows("logits", logits)
    if teacher_values is None:
        raise SfcError("teacher_values is required")
    check_packed(logits, temperature, teacher_ids, lengths, teacher_values)
    if temperature.requires_grad or teacher_values.requires_grad or getattr(forward_ad, "_current_level", 0) >= 0:
        check_derivatives(logits, temperature=temperature, teacher_values=teacher_values)
    if torch.is_grad_enabled() and logits.requires_grad:
        _, context = _enter(logits.device, stream, logits, temperature, teacher_ids, teacher_values, lengths)
        with context:
            return DistillOutput(*_Distill.apply(logits, row, temperature, teacher_ids, teacher_values, lengths, bool(normalise)))
    loss, _, status = _distill_forward(logits, row, temperature, teacher_ids, teacher_values, lengths, normalise, stream, False)
    return DistillOutput(loss, status)


def distill_loss_and_grad(logits, temperature, teacher_ids, teacher_values, lengths, grad_loss, normalise: bool = False,
                          grad=None, stream=None, test_stall: bool = False) -> DistillGradOutput:
    """``distill_loss`` and its gradient in one call, for a known upstream gradient ``grad_loss`` [B] f32 (a mean
    over the batch: 1 / B each): the logits are read once. ``grad`` may give the [B, V] tensor to write (not the
    logits themselves). Outside autograd."""
    row = check_rows("logits", logits)
    if teacher_values is None:
        raise SfcError("teacher_values is required")
    dev, B, _ = check_packed(logits, temperature, teacher_ids, lengths, teacher_values)
    _expect("grad_loss", grad_loss, dev, torch.float32, numel=B)
    grad_row = logits.shape[1] if grad is None else _check_grad(grad, logits)
    stream, context = _enter(dev, stream, logits, temperature, teacher_ids, teacher_values, lengths, grad_loss, grad)
    with context:
        loss = torch.empty(B, dtype=torch.float32, device=dev)
        status = torch.empty(B, dtype=torch.int32, device=dev)
        if grad is None:
            grad = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        rc = load_library().sfc_distill_forward_backward(
            *_rows_args(logits, row, temperature), *_teacher_args(teacher_ids, teacher_values, lengths, normalise, FLAG_TEST_STALL if test_stall else 0),
            grad_loss.data_ptr(), loss.data_ptr(), status.data_ptr(), grad.data_ptr(), grad_row, stream)
    if rc != SFC_OK:
        _raise("sfc_distill_forward_backward", rc)
    return DistillGradOutput(loss, grad, status)


def replay_logprob_backward(logits, temperature, support_ids, lengths, tokens, grad_token_logprob,
                            grad_support_logprobs=None, grad=None, stream=None):
    """The gradient of ``replay_logprob`` with respect to ``logits`` [B, V], from the upstream gradients
    ``grad_token_logprob`` [B] f32 and, where it is given, ``grad_support_logprobs`` [B, W] f32: a dense
    [B, V] tensor of the logits' dtype, zero outside the supports (written into ``grad`` when that is given)."""
    row = check_rows("logits", logits)
    dev, B, W = check_packed(logits, temperature, support_ids, lengths, grad_support_logprobs, "grad_support_logprobs", "support_ids")
    _expect("tokens", tokens, dev, torch.int32, numel=B)
    _expect("grad_token_logprob", grad_token_logprob, dev, torch.float32, numel=B)
    grad_row = logits.shape[1] if grad is None else _check_grad(grad, logits)
    stream, context = _enter(dev, stream, logits, temperature, support_ids, lengths, tokens, grad_token_logprob,
                             grad_support_logprobs, grad)
    with context:
        if grad is None:
            grad = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        rc = load_library().sfc_replay_backward(
            *_rows_args(logits, row, temperature), support_ids.data_ptr(), lengths.data_ptr(), W, tokens.data_ptr(),
            grad_token_logprob.data_ptr(), _ptr(grad_support_logprobs), grad.data_ptr(), grad_row, stream)
    if rc != SFC_OK:
        _raise("sfc_replay_backward", rc)
    return grad


class _Replay(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, temperature, support_ids, lengths, tokens, support_logprobs):
        out = replay_logprob(logits.detach(), temperature, support_ids, lengths, tokens, support_logprobs)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(logits, temperature, support_ids, lengths, tokens)
        ctx.mark_non_differentiable(out.row_status)
        return out.token_logprob, out.support_logprobs, out.row_status

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_token, grad_entries, _):
        logits, temperature, support_ids, lengths, tokens = ctx.saved_tensors
        if grad_token is None and grad_entries is None:
            return (None,) * 6
        grad_token = torch.zeros_like(temperature) if grad_token is None else grad_token.to(torch.float32).contiguous()
        if grad_entries is not None:
            grad_entries = grad_entries.to(torch.float32).contiguous()
        grad = replay_logprob_backward(logits.detach(), temperature, support_ids, lengths, tokens, grad_token, grad_entries)
        return grad, None, None, None, None, None


def differentiable_replay(logits, temperature, support_ids, lengths, tokens, support_logprobs, stream) -> ReplayOutput:
    check_rows("logits", logits)
    check_derivatives(logits, temperature=temperature)
    _, context = _enter(logits.device, stream, logits, temperature, support_ids, lengths, tokens)
    with context:
        return ReplayOutput(*_Replay.apply(logits, temperature, support_ids, lengths, tokens, support_logprobs))
