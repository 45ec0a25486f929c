"""Verification of drafted tokens against the target's distributions: over full logit rows, and over captured
supports (the filtered distributions that the decode step captured).

Like the rest of the binding this only checks and marshals arguments (include/sfc.h has the rule).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import (FLAG_GREEDY_T0, MAX_DRAFTS, MAX_PACKED_WIDTH, SFC_OK, SfcError, _Workspaces, _check_tensor, _dtype_code, _enter, _expect,
               _ptr, load_library, strerror)


class VerifyOutput(NamedTuple):
    accepted: "object"  # int32 [B]
    tokens: "object"  # int32 [B, D + 1]: the accepted drafts, the drawn token, then -1
    token_logprobs: "object"  # float32 [B, D + 1]
    row_status: "object"  # int32 [B]


_workspaces = _Workspaces("verify_workspace_size")


def verify_workspace_size(B: int, D: int, V: int, dtype: int) -> int:
    """Bytes of workspace that ``verify_drafts`` needs: zero-filled before its first use, one call at a time."""
    return int(load_library().sfc_verify_workspace_size(B, D, V, dtype))


def check_positions(name, t, B, positions):
    """[B, positions, V] logits whose rows are contiguous (the rows may lie anywhere: they are only read);
    returns (V, request stride, row stride)."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != B or shape[1] != positions or shape[2] < 1:
        raise SfcError(f"{name} must be [{B}, {positions}, V], got {tuple(shape)}")
    _dtype_code(t)
    V, (request, row, one) = shape[2], t.stride()
    if one != 1 and V > 1:
        raise SfcError(f"{name} rows must be contiguous")
    return V, request, row


def check_drafts(draft_tokens, uniforms, num_drafts, device):
    """[B, D] drafted tokens and uniforms, [B] counts; returns (B, D)."""
    shape = draft_tokens.shape
    if len(shape) != 2 or shape[0] < 1:
        raise SfcError("draft_tokens must be a non-empty [B, D] tensor")
    B, D = shape
    if D < 1 or D > MAX_DRAFTS:
        raise SfcError(f"draft_tokens must hold 1 to {MAX_DRAFTS} drafts a request, got {D}")
    _expect("draft_tokens", draft_tokens, device, torch.int32)
    _expect("uniforms", uniforms, device, torch.float32, shape)
    if num_drafts is not None:
        _expect("num_drafts", num_drafts, device, torch.int32, numel=B)
    return B, D


def _outputs(B, D, dev):
    empty, i32 = torch.empty, torch.int32
    return VerifyOutput(empty(B, dtype=i32, device=dev), empty((B, D + 1), dtype=i32, device=dev),
                        empty((B, D + 1), dtype=torch.float32, device=dev), empty(B, dtype=i32, device=dev))


_U64 = 0xFFFFFFFFFFFFFFFF


def verify_drafts(target_logits, draft_logits, draft_tokens, uniforms, temperature, seed: int, step: int,
                  draft_temperature=None, num_drafts=None, greedy_t0: bool = False, row_offset: int = 0, workspace=None,
                  stream=None) -> VerifyOutput:
    """Accept or refuse ``draft_tokens`` [B, D] int32 against ``target_logits`` [B, D + 1, V] (bf16/f32 CUDA) and
    draw the token that follows. ``draft_logits`` [B, D, V] are the rows that the drafts were drawn from, None for
    drafts that were not drawn (looked up); ``uniforms`` [B, D] f32 in [0, 1) decide; ``temperature`` [B] f32 (and
    ``draft_temperature``, the same when omitted); ``num_drafts`` [B] int32 for requests with fewer than D drafts;
    ``greedy_t0`` makes rows of temperature 0 greedy; ``seed``, ``step`` and ``row_offset`` key the draw's noise.
    The workspace may be omitted: the binding then keeps one per device and stream, and one for each graph capture on it
    (after a call on that stream outside the capture). See include/sfc.h."""
    if not target_logits.is_cuda:
        raise SfcError(f"target_logits must be a CUDA tensor, got {target_logits.device}")
    dev = target_logits.device
    B, D, V, strides = check_verify_layout(target_logits, draft_logits, draft_tokens, uniforms, temperature, draft_temperature,
                                           num_drafts)
    dt = _dtype_code(target_logits)
    lib = load_library()
    stream, context = _enter(dev, stream, target_logits, draft_logits, draft_tokens, uniforms, temperature, draft_temperature,
                             num_drafts, workspace)
    with context:
        if workspace is None:
            workspace = _workspaces.get(lib.sfc_verify_workspace_size(B, D, V, dt), dev, stream)
        else:
            _check_tensor("workspace", workspace, dev, workspace.dtype)
        out = _outputs(B, D, dev)
        rc = lib.sfc_verify_drafts(
            target_logits.data_ptr(), _ptr(draft_logits), dt, B, D, V, *strides, temperature.data_ptr(), _ptr(draft_temperature),
            draft_tokens.data_ptr(), _ptr(num_drafts), uniforms.data_ptr(), seed & _U64, step & _U64, row_offset,
            FLAG_GREEDY_T0 if greedy_t0 else 0, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(),
            workspace.data_ptr(), workspace.nbytes, stream)
    if rc != SFC_OK:
        raise SfcError(f"sfc_verify_drafts: {strerror(rc)} ({rc})")
    return out


def check_verify_layout(target_logits, draft_logits, draft_tokens, uniforms, temperature, draft_temperature, num_drafts):
    """The host-side checks of ``verify_drafts``; returns (B, D, V, the four strides)."""
    dev = target_logits.device
    B, D = check_drafts(draft_tokens, uniforms, num_drafts, dev)
    V, request, row = check_positions("target_logits", target_logits, B, D + 1)
    strides = [request, row, 0, 0]
    if draft_logits is not None:
        if draft_logits.device != dev or draft_logits.dtype != target_logits.dtype:
            raise SfcError("draft_logits must have the target logits' device and dtype")
        Vd, strides[2], strides[3] = check_positions("draft_logits", draft_logits, B, D)
        if Vd != V:
            raise SfcError(f"draft_logits must have the target's vocabulary of {V}, got {Vd}")
    if temperature is None:
        raise SfcError("temperature is required")
    _expect("temperature", temperature, dev, torch.float32, numel=B)
    if draft_temperature is not None:
        _expect("draft_temperature", draft_temperature, dev, torch.float32, numel=B)
    return B, D, V, strides


def verify_supports(target_ids, target_logprobs, target_lengths, draft_ids, draft_logprobs, draft_lengths, draft_tokens,
                    uniforms, seed: int, step: int, num_drafts=None, row_offset: int = 0, stream=None) -> VerifyOutput:
    """``verify_drafts`` over captured supports: ``target_ids`` / ``target_logprobs`` [B, D + 1, W] and
    ``target_lengths`` [B, D + 1] as the decode step wrote them for the target's rows, ``draft_*`` [B, D, Wd] and
    [B, D] for the draft's (None, or a length of 0: a draft that was not drawn). See include/sfc.h."""
    if not target_ids.is_cuda:
        raise SfcError(f"target_ids must be a CUDA tensor, got {target_ids.device}")
    dev = target_ids.device
    B, D, W, Wd = check_supports_layout(target_ids, target_logprobs, target_lengths, draft_ids, draft_logprobs, draft_lengths,
                                        draft_tokens, uniforms, num_drafts)
    lib = load_library()
    stream, context = _enter(dev, stream, target_ids, target_logprobs, target_lengths, draft_ids, draft_logprobs, draft_lengths,
                             draft_tokens, uniforms, num_drafts)
    with context:
        out = _outputs(B, D, dev)
        rc = lib.sfc_verify_supports(
            target_ids.data_ptr(), target_logprobs.data_ptr(), target_lengths.data_ptr(), W, _ptr(draft_ids), _ptr(draft_logprobs),
            _ptr(draft_lengths), Wd, B, D, draft_tokens.data_ptr(), _ptr(num_drafts), uniforms.data_ptr(), seed & _U64, step & _U64,
            row_offset, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), stream)
    if rc != SFC_OK:
        raise SfcError(f"sfc_verify_supports: {strerror(rc)} ({rc})")
    return out


def check_supports_layout(target_ids, target_logprobs, target_lengths, draft_ids, draft_logprobs, draft_lengths, draft_tokens,
                          uniforms, num_drafts):
    """The host-side checks of ``verify_supports``; returns (B, D, the target's width, the draft's or 0)."""
    dev = target_ids.device
    B, D = check_drafts(draft_tokens, uniforms, num_drafts, dev)
    W = _check_supports(_TARGET, target_ids, target_logprobs, target_lengths, B, D + 1, dev)
    return B, D, W, 0 if draft_ids is None else _check_supports(_DRAFT, draft_ids, draft_logprobs, draft_lengths, B, D, dev)


_TARGET = ("target_ids", "target_logprobs", "target_lengths")
_DRAFT = ("draft_ids", "draft_logprobs", "draft_lengths")


def _check_supports(names, ids, lps, lengths, B, positions, dev):
    shape = ids.shape
    if len(shape) != 3 or shape[0] != B or shape[1] != positions or lps is None or lengths is None:
        raise SfcError(f"{names[0]} and {names[1]} must be [{B}, {positions}, W], {names[2]} [{B}, {positions}]")
    W = shape[2]
    if W < 1 or W > MAX_PACKED_WIDTH:
        raise SfcError(f"{names[0]} must be 1 to {MAX_PACKED_WIDTH} wide, got {W}")
    _expect(names[0], ids, dev, torch.int32)
    _expect(names[1], lps, dev, torch.float32, shape)
    _expect(names[2], lengths, dev, torch.int32, (B, positions))
    return W
