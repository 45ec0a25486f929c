"""Gradient norms and clipping at the ends of their ranges."""
import ctypes
import os

import numpy as np
import pytest

import oracle
import top_support_capture_gb300 as sfc
from top_support_capture_gb300 import gradients

torch = pytest.importorskip("torch")
FAR = 1 << 40  # never dereferenced: the checks reject the call first


@pytest.mark.parametrize("count,dtype,fine", [(2 ** 43, 1, True), (2 ** 43, 0, True), (2 ** 43 + 1, 1, False), (2 ** 44, 1, False), (2 ** 44, 0, False)])
def test_most_elements(count, dtype, fine):
    """Chunks of 2^13 f32 elements are counted in 32 bits, one more for each tensor."""
    if not os.path.exists(sfc.library_path()):
        from top_support_capture_gb300 import build

        build.build()
    lib = sfc.load_library()
    rc = lib.sfc_grad_norm((ctypes.c_void_p * 1)(FAR), (ctypes.c_int64 * 1)(count), (ctypes.c_int32 * 1)(dtype), 1, FAR, None, 0, None)
    assert rc == (sfc.SFC_EWORKSPACE if fine else sfc.SFC_EINVAL)


def test_wrong_types_are_named():
    for name in ("grads", "out"):
        for others in ([], [torch.zeros(2)]):
            with pytest.raises(sfc.SfcError, match=f"{name} must be bfloat16 or float32"):
                gradients._arrays([*others, torch.zeros(3, dtype=torch.float16)], name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes", [[5000, 33], [1_000_001, 7]])
@pytest.mark.parametrize("size,max_norm", [(1e37, 1.0), (1e37, 1e-3), (3e37, 1e-6), (1e30, 1e-12), (1e30, 1e12), (1e37, 0.0)])
def test_scales_below_the_smallest_normal_number(dtype, out, sizes, size, max_norm):
    """Clipped elements are ordinary numbers where the scale is a subnormal one. Tolerance as in test_grad_norm_gpu: 20 half steps,
    the rounding to the output's type, half of the smallest number."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gen = torch.Generator("cuda").manual_seed(1)
    # starting one element into their buffers: eights at a time and, into outputs that start at a boundary, one by one
    grads = [(torch.randn(n + 1, generator=gen, device="cuda") * size).to(dtype)[1:] for n in sizes]
    before = [t.double().cpu().numpy() for t in grads]
    want = oracle.clip_scale(oracle.grad_norm(before), max_norm)
    to = grads if out is None else [torch.empty(n, dtype=out, device="cuda") for n in sizes]
    sfc.clip_grad_norm(grads, max_norm, out=None if out is None else to)
    for b, o in zip(before, to):
        bf16 = o.dtype == torch.bfloat16
        limit = (20 * 2.0 ** -24 + (2.0 ** -8 if bf16 else 2.0 ** -24)) * np.abs(b * want) + (2.0 ** -134 if bf16 else 2.0 ** -149)
        assert np.all(np.abs(o.double().cpu().numpy() - b * want) <= limit)
