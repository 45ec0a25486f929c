"""The global norm of a model's gradients and their clipping, over any number of tensors in one or two launches.

Like the rest of the binding this only checks and marshals arguments (include/sfc.h has the formulas)."""
from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad

from . import SFC_OK, SfcError, _dtype_code, _enter, load_library
from .training import _raise


def _dense(t):
    """Whether the tensor's elements fill their memory without gaps or overlaps, in whatever order."""
    expected = 1
    for stride, size in sorted((stride, size) for size, stride in zip(t.shape, t.stride()) if size != 1):
        if stride != expected:
            return False
        expected *= size
    return True


def check_tensors(name, tensors):
    """The tensors as a list (entries None left out), each on one CUDA device and dense."""
    tensors = [t for t in ([tensors] if isinstance(tensors, torch.Tensor) else tensors) if t is not None]
    if not tensors:
        raise SfcError(f"{name} holds no tensor")
    device = tensors[0].device
    if device.type != "cuda":
        raise SfcError(f"{name} must be CUDA tensors, got {device}")
    check_layouts(name, tensors, device)
    return tensors


def check_layouts(name, tensors, device):
    derivatives, dual = torch.is_grad_enabled(), getattr(forward_ad, "_current_level", 0) >= 0
    for i, t in enumerate(tensors):
        if t.device != device:
            raise SfcError(f"{name}[{i}] must be on {device}, got {t.device}")
        if t.layout is not torch.strided:
            raise SfcError(f"{name}[{i}] must be a dense tensor, got {t.layout}")
        if not t.is_contiguous() and t.numel() > 0 and not _dense(t):
            raise SfcError(f"{name}[{i}] must fill its memory without gaps (make it contiguous)")
        if derivatives and t.requires_grad:
            raise SfcError(f"{name}[{i}] requires a gradient, which is not given: detach it")
        if dual and forward_ad.unpack_dual(t).tangent is not None:
            raise SfcError(f"{name}[{i}] is a forward-mode dual tensor: there is no forward-mode derivative")


def _arrays(tensors):
    n = len(tensors)
    return ((ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors]), (ctypes.c_int64 * n)(*[t.numel() for t in tensors]),
            (ctypes.c_int32 * n)(*[_dtype_code(t) for t in tensors]))


def grad_norm(grads, stream=None):
    """The global norm of ``grads`` (an iterable of bf16/f32 CUDA tensors of one device, entries None left out): a float32
    scalar tensor. See include/sfc.h."""
    grads = check_tensors("grads", grads)
    return _run(grads, None, 0.0, stream)


def clip_grad_norm(grads, max_norm: float, out=None, stream=None):
    """Scales ``grads`` so that their global norm is at most ``max_norm``, in place, or into the tensors of ``out`` (as many,
    of the same shapes; bf16 or f32 each, as the optimizer wants them). Returns the norm before clipping, a float32 scalar
    tensor. No host synchronisation. See include/sfc.h."""
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise SfcError(f"max_norm must be >= 0, got {max_norm}")
    grads = check_tensors("grads", grads)
    if out is not None:
        out = check_tensors("out", out)
        check_out(grads, out)
    return _run(grads, grads if out is None else out, max_norm, stream)


def check_out(grads, out):
    if len(out) != len(grads):
        raise SfcError(f"out must hold {len(grads)} tensors, got {len(out)}")
    for i, (g, o) in enumerate(zip(grads, out)):
        if o.device != g.device or o.shape != g.shape or (o.stride() != g.stride() and not (o.is_contiguous() and g.is_contiguous())):
            raise SfcError(f"out[{i}] must have grads[{i}]'s device, shape and strides")


def _run(grads, out, max_norm, stream):
    lib, dev, n = load_library(), grads[0].device, len(grads)
    addresses, counts, dtypes = _arrays(grads)
    stream, context = _enter(dev, stream, *grads, *(out if out is not None and out is not grads else ()))
    with context:
        norm = torch.empty((), dtype=torch.float32, device=dev)
        # the CTAs' sums: memory of this call alone, so calls and captured graphs that run side by side share none
        nbytes = lib.sfc_grad_norm_workspace_size(n)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        if out is None:
            rc = lib.sfc_grad_norm(addresses, counts, dtypes, n, norm.data_ptr(), workspace.data_ptr(), nbytes, stream)
        else:
            to, _, to_dtypes = (addresses, counts, dtypes) if out is grads else _arrays(out)
            rc = lib.sfc_clip_grad_norm(addresses, counts, dtypes, n, max_norm, to, to_dtypes, norm.data_ptr(), workspace.data_ptr(),
                                        nbytes, stream)
    if rc != SFC_OK:
        _raise("sfc_grad_norm" if out is None else "sfc_clip_grad_norm (tensors that overlap?)", rc)
    if out is not None:  # autograd's view of what was written
        for t in out:
            if not t.is_inference():
                torch.autograd.graph.increment_version(t)
    return norm
