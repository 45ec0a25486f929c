"""Gradient norms and clipping at the ends of their ranges."""
import ctypes
import os

import pytest

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
