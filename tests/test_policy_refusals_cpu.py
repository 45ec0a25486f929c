"""Refusals of the whole-vocabulary calls and of gradient clipping: the C ABI's host checks (they run before any CUDA call,
so no GPU is needed) and the binding's tensor checks on CPU tensors."""
import ctypes
import os
import re

import pytest

import top_support_capture_gb300 as sfc
from top_support_capture_gb300 import gradients, policy

torch = pytest.importorskip("torch")
fwAD = torch.autograd.forward_ad
FAKE = 1 << 20  # never dereferenced: the checks reject the call first
FAR = 1 << 40   # a second array that does not overlap the first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sfc.library_path()):
        from top_support_capture_gb300 import build

        build.build()
    return sfc.load_library()


ROWS = dict(logits=FAKE, dtype=0, B=4, V=16, stride=16, T=FAKE)
ROW_FAULTS = [dict(logits=None), dict(dtype=7), dict(B=0), dict(B=2 ** 31), dict(V=0), dict(V=2 ** 31), dict(stride=15), dict(T=None),
              dict(logits=FAKE + 1), dict(dtype=1, logits=FAKE + 2)]
GRAD_FAULTS = [dict(grad=None), dict(grad=FAR + 1), dict(grad_stride=15), dict(grad=FAKE), dict(grad=FAKE + 64), dict(grad=FAKE - 64)]


@pytest.mark.parametrize("fault", ROW_FAULTS + [dict(M=-1), dict(M=sfc.MAX_GIVEN + 1), dict(tokens=None), dict(lps=None), dict(top=-1),
                                                dict(top=sfc.MAX_TOP + 1), dict(top_ids=None), dict(top_lps=None), dict(entropy=None),
                                                dict(stats=FAKE + 4), dict(status=None)])
def test_token_logprobs(lib, fault):
    a = {**ROWS, "tokens": FAKE, "M": 2, "top": 3, "lps": FAKE, "entropy": FAKE, "top_ids": FAKE, "top_lps": FAKE, "stats": None,
         "status": FAKE, "stream": None, **fault}
    assert lib.sfc_token_logprobs(*a.values()) == sfc.SFC_EINVAL


@pytest.mark.parametrize("fault", ROW_FAULTS + GRAD_FAULTS + [dict(M=-1), dict(M=sfc.MAX_GIVEN + sfc.MAX_TOP + 1), dict(tokens=None),
                                                              dict(stats=None), dict(stats=FAKE + 8)])
def test_token_logprobs_backward(lib, fault):
    a = {**ROWS, "tokens": FAKE, "M": 2, "stats": FAKE, "g": FAKE, "h": None, "grad": FAR, "grad_stride": 16, "stream": None, **fault}
    assert lib.sfc_token_logprobs_backward(*a.values()) == sfc.SFC_EINVAL


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("fault", ROW_FAULTS + GRAD_FAULTS + [dict(tokens=None), dict(A=None), dict(up=None), dict(loss=None), dict(lps=None),
                                                              dict(entropy=None), dict(status=None), dict(low=-0.1), dict(low=1.5),
                                                              dict(low=NAN), dict(high=-0.1), dict(high=INF), dict(high=NAN),
                                                              dict(weight=NAN), dict(weight=INF), dict(flags=1)])
def test_policy(lib, fault):
    a = {**ROWS, "tokens": FAKE, "old": None, "A": FAKE, "low": 0.2, "high": 0.2, "weight": 0.0, "flags": 0, "up": FAKE, "loss": FAKE,
         "lps": FAKE, "entropy": FAKE, "status": FAKE, "grad": FAR, "grad_stride": 16, "stream": None, **fault}
    assert lib.sfc_policy_forward_backward(*a.values()) == sfc.SFC_EINVAL


def clip(lib, grads, out, counts, dtypes=(0, 1), out_dtypes=(0, 1), n=2, max_norm=1.0, norm=FAKE, ws=FAKE, ws_bytes=1 << 20):
    p = lambda v: None if v is None else (ctypes.c_void_p * len(v))(*v)
    i32 = lambda v: None if v is None else (ctypes.c_int32 * len(v))(*v)
    counts = None if counts is None else (ctypes.c_int64 * len(counts))(*counts)
    return lib.sfc_clip_grad_norm(p(grads), counts, i32(dtypes), n, max_norm, p(out), i32(out_dtypes), norm, ws, ws_bytes, None)


A, B, C, D = (FAR + (i << 30) for i in range(4))
CLIP = dict(grads=[A, B], out=[C, D], counts=[100, 10])


@pytest.mark.parametrize("fault", [
    dict(grads=None), dict(counts=None), dict(dtypes=None), dict(out=None), dict(out_dtypes=None), dict(n=-1), dict(n=2 ** 20 + 1),
    dict(counts=[-1, 10]), dict(counts=[2 ** 44, 1]), dict(counts=[2 ** 60, 1]), dict(dtypes=(0, 2)), dict(out_dtypes=(3, 1)),
    dict(grads=[None, B]), dict(out=[None, D]), dict(grads=[A + 1, B]), dict(grads=[A, B + 2]), dict(out=[C + 1, D]), dict(out=[C, D + 2]),
    dict(max_norm=-1.0), dict(max_norm=NAN), dict(norm=None), dict(ws=FAKE + 4),
    # what is written shares bytes: with another output, another tensor, its own tensor elsewhere or in another type
    dict(out=[C, C]), dict(out=[C, C + 196]), dict(out=[B, D]), dict(out=[C, A]), dict(out=[A + 2, D]), dict(out=[A, D], out_dtypes=(1, 1)),
    dict(grads=[A, A], out=[A, A], dtypes=(0, 0), out_dtypes=(0, 0)), dict(grads=[A, A + 196], out=[A, A + 196]),
    dict(grads=[A, A], out=[C, A], dtypes=(1, 1)),
])
def test_clip(lib, fault):
    assert clip(lib, **{**CLIP, **fault}) == sfc.SFC_EINVAL


def test_clip_workspace(lib):
    need = lib.sfc_grad_norm_workspace_size(2)
    assert need > 0 and lib.sfc_grad_norm_workspace_size(5000) > need
    assert lib.sfc_grad_norm_workspace_size(-1) == 0 and lib.sfc_grad_norm_workspace_size(2 ** 20 + 1) == 0
    # (these reach the workspace check: all before it is in order, neighbours that touch among it)
    for fine in ({}, dict(out=[A, B]), dict(out=[C, C + 200]), dict(grads=[A, A + 200], out=[A, A + 200]), dict(grads=[A, A]),
                 dict(counts=[0, 10], grads=[None, B], out=[None, D]), dict(max_norm=INF)):
        assert clip(lib, **{**CLIP, **fine}, ws=None) == sfc.SFC_EWORKSPACE
        assert clip(lib, **{**CLIP, **fine}, ws_bytes=need - 1) == sfc.SFC_EWORKSPACE


def test_constants_match_the_header():
    src = open(os.path.join(os.path.dirname(__file__), "..", "include", "sfc.h")).read()
    consts = dict(re.findall(r"#define (SFC_[A-Z_0-9]+) \(?(-?\d+)u?\)?", src))
    assert int(consts["SFC_MAX_GIVEN"]) == sfc.MAX_GIVEN and int(consts["SFC_MAX_TOP"]) == sfc.MAX_TOP


def test_token_layouts():
    x, i32 = torch.zeros(3, 10), torch.int32
    assert policy.check_tokens(x, None) == 0 and policy.check_tokens(x, torch.zeros(3, dtype=i32)) == 1
    assert policy.check_tokens(x, torch.zeros(3, 64, dtype=i32)) == 64
    for bad in (torch.zeros(2, dtype=i32), torch.zeros(3, dtype=torch.int64), torch.zeros(3, 65, dtype=i32), torch.zeros(3, 0, dtype=i32),
                torch.zeros(3, 1, 1, dtype=i32), torch.zeros((), dtype=i32), torch.zeros(2, 3, dtype=i32).t()):
        with pytest.raises(sfc.SfcError):
            policy.check_tokens(x, bad)
    with pytest.raises(sfc.SfcError, match="CUDA"):
        sfc.token_logprobs(x, torch.ones(3))
    with pytest.raises(sfc.SfcError, match="CUDA"):
        sfc.policy_loss_and_grad(x, torch.ones(3), torch.zeros(3, dtype=i32), torch.ones(3), torch.ones(3))


def test_tensor_lists():
    cpu = torch.device("cpu")
    f = lambda *t: gradients.check_layouts("grads", list(t), cpu)
    f(torch.zeros(3, 4), torch.zeros(4, 3).t(), torch.zeros(()), torch.zeros(0), torch.zeros(2, 3, 4).permute(2, 0, 1), torch.zeros(5, 1, 3)[:, :1])
    for bad in (torch.zeros(3, 8)[:, :4], torch.zeros(4).expand(3, 4), torch.zeros(10)[::2], torch.zeros(3, 4, requires_grad=True),
                torch.sparse_coo_tensor([[0]], [1.0], (3,))):
        with pytest.raises(sfc.SfcError, match=r"grads\[1\]"):
            f(torch.zeros(3), bad)
    with torch.no_grad():
        f(torch.zeros(3, 4, requires_grad=True))
    with fwAD.dual_level(), pytest.raises(sfc.SfcError, match="forward-mode"):
        f(fwAD.make_dual(torch.zeros(3), torch.ones(3)))
    for empty in ([], [None, None]):
        with pytest.raises(sfc.SfcError, match="no tensor"):
            sfc.grad_norm(empty)
    with pytest.raises(sfc.SfcError, match="CUDA"):
        sfc.grad_norm([torch.zeros(3)])
    for bad in (-1.0, NAN):
        with pytest.raises(sfc.SfcError, match="max_norm"):
            sfc.clip_grad_norm([torch.zeros(3)], bad)
    with pytest.raises(sfc.SfcError, match="bfloat16 or float32"):
        gradients._arrays([torch.zeros(3, dtype=torch.float16)])
    a, b = torch.zeros(3, 4), torch.zeros(4, 3).t()
    gradients.check_out([a, b], [torch.zeros(3, 4, dtype=torch.bfloat16), torch.zeros(4, 3).t()])
    for out in ([a], [b, b], [a, torch.zeros(3, 4)], [a, torch.zeros(12)]):
        with pytest.raises(sfc.SfcError, match="out"):
            gradients.check_out([a, b], out)
