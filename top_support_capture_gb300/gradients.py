"""The global norm of a model's gradients and their clipping, over any number of tensors in one or two launches.

Like the rest of the binding this only checks and marshals arguments (include/sfc.h has the formulas)."""
from __future__ import annotations

from array import array
from operator import attrgetter

import torch
from torch.autograd import forward_ad

from . import SFC_BF16, SFC_F32, SFC_OK, SfcError, _enter, load_library
from .training import _raise

_dtype, _requires_grad = attrgetter("dtype"), attrgetter("requires_grad")
_Tensor = torch.Tensor


def _dense(t):
    """Whether the tensor's elements fill their memory without gaps or overlaps, in whatever order."""
    expected = 1
    for stride, size in sorted((stride, size) for size, stride in zip(t.shape, t.stride()) if size != 1):
        if stride != expected:
            return False
        expected *= size
    return True


def _listed(tensors):
    return [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)


def pair(grads, out):
    """The gradients that there are (entries None left out) and each one's output: the entry in its place of an ``out`` that is as
    long as ``grads``, or of one that has an entry for each gradient there is."""
    grads, out = _listed(grads), _listed(out)
    there, places = [g for g in grads if g is not None], range(len(out))
    if len(out) == len(grads):
        if len(there) < len(grads):
            places = [i for i in places if grads[i] is not None]
            out = [out[i] for i in places]
    elif len(out) != len(there):
        raise SfcError(f"out must hold {len(grads)} tensors" + (f" (or {len(there)}, one for each gradient there is)" if len(there) < len(grads) else "")
                       + f", got {len(out)}")
    if len([o for o in out if o is not None]) < len(out):
        raise SfcError(f"out[{next(i for i, o in zip(places, out) if o is None)}] is None beside a gradient")
    return there, out


def check_tensors(name, tensors):
    """The tensors as a list (entries None left out), each on one CUDA device and dense; and whether all are contiguous."""
    tensors = [t for t in _listed(tensors) if t is not None]
    return tensors, check_listed(name, tensors)


def check_listed(name, tensors):
    if not tensors:
        raise SfcError(f"{name} holds no tensor")
    if _all_plain(tensors):
        return True
    device = tensors[0].device
    if device.type != "cuda":
        raise SfcError(f"{name} must be CUDA tensors, got {device}")
    check_layouts(name, tensors, device)
    return False


def _all_plain(tensors):
    """Whether there is nothing to look at one by one. The calls over many small tensors take as long as their Python: what
    is asked of every tensor is asked by one map."""
    try:
        devices = set(map(_Tensor.get_device, tensors))
        return (len(devices) == 1 and devices.pop() >= 0 and all(map(_Tensor.is_contiguous, tensors))
                and not (torch.is_grad_enabled() and any(map(_requires_grad, tensors))) and getattr(forward_ad, "_current_level", 0) < 0)
    except RuntimeError:  # (a tensor without strides)
        return False


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


_CODES = {torch.bfloat16: SFC_BF16, torch.float32: SFC_F32}


def _arrays(tensors, name="grads"):
    """(addresses, counts, dtype codes) as the library reads them."""
    dtypes = list(map(_dtype, tensors))
    try:
        if dtypes.count(dtypes[0]) == len(dtypes):
            codes = array("i", [_CODES[dtypes[0]]]) * len(dtypes)
        else:
            codes = array("i", map(_CODES.__getitem__, dtypes))
    except KeyError as e:
        raise SfcError(f"{name} must be bfloat16 or float32, got {e.args[0]}") from None
    return array("Q", map(_Tensor.data_ptr, tensors)), array("q", map(_Tensor.numel, tensors)), codes


def grad_norm(grads, stream=None):
    """The global norm of ``grads`` (an iterable of bf16/f32 CUDA tensors of one device, entries None left out): a float32
    scalar tensor. See include/sfc.h."""
    grads, _ = check_tensors("grads", grads)
    return _run(grads, _arrays(grads), None, None, 0.0, stream)


def clip_grad_norm(grads, max_norm: float, out=None, stream=None):
    """Scales ``grads`` so that their global norm is at most ``max_norm``, in place, or into the tensors of ``out`` (each of as many
    elements as its gradient; bf16 or f32, as the optimizer wants them). Beside entries None of ``grads`` ``out`` may be as long as
    they are, then its entries there are left alone, or have one entry for each gradient there is. Returns the norm before
    clipping, a float32 scalar tensor. No host synchronisation. See include/sfc.h."""
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise SfcError(f"max_norm must be >= 0, got {max_norm}")
    if out is None:
        grads, _ = check_tensors("grads", grads)
        lists = _arrays(grads)
        return _run(grads, lists, grads, lists, max_norm, stream)
    grads, out = pair(grads, out)
    plain, out_plain = check_listed("grads", grads), check_listed("out", out)
    lists, to = _arrays(grads), _arrays(out, "out")
    if to[1] != lists[1] or out[0].device != grads[0].device or not (plain and out_plain):
        check_out(grads, out)
    return _run(grads, lists, out, to, max_norm, stream)


def check_out(grads, out):
    """Each of ``out`` beside its gradient: of as many elements in the same order (contiguous both, or the same layout)."""
    if len(out) != len(grads):
        raise SfcError(f"out must hold {len(grads)} tensors, got {len(out)}")
    for i, (g, o) in enumerate(zip(grads, out)):
        if o.device != g.device or o.numel() != g.numel():
            raise SfcError(f"out[{i}] must be on grads[{i}]'s device and have its shape")
        if not (o.is_contiguous() and g.is_contiguous()) and (o.shape != g.shape or o.stride() != g.stride()):
            raise SfcError(f"out[{i}] must have grads[{i}]'s shape and strides (or both be contiguous)")


def _run(grads, lists, out, to, max_norm, stream):
    lib, dev, n = load_library(), grads[0].device, len(grads)
    stream, context = _enter(dev, stream, *grads, *(out if out is not None and out is not grads else ()))
    with context:
        nbytes = lib.sfc_grad_norm_workspace_size(n)
        norm = torch.empty((), dtype=torch.float32, device=dev)
        # the CTAs' sums: memory of this call alone, so calls and captured graphs that run side by side share none
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        address = lambda a: a.buffer_info()[0]  # (the arrays live until the call is over)
        tail = norm.data_ptr(), workspace.data_ptr(), nbytes, stream
        rc = (lib.sfc_grad_norm(*map(address, lists), n, *tail) if out is None else
              lib.sfc_clip_grad_norm(*map(address, lists), n, max_norm, address(to[0]), address(to[2]), *tail))
    if rc != SFC_OK:
        _raise("sfc_grad_norm" if out is None else "sfc_clip_grad_norm (tensors that overlap?)", rc)
    if out is not None:  # autograd's view of what was written
        torch.autograd.graph.increment_version(out)
    return norm
