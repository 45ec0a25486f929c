"""Refusals of the distillation, replay-gradient and verification calls: the C ABI's host checks (they run
before any CUDA call, so no GPU is needed) and the binding's tensor checks on CPU tensors."""
import os

import pytest

import top_support_capture_gb300 as sfc
from top_support_capture_gb300 import speculative, training

torch = pytest.importorskip("torch")
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
TEACHER = dict(ids=FAKE, values=FAKE, lengths=FAKE, W=8, flags=0)
TEACHER_FAULTS = [dict(ids=None), dict(values=None), dict(lengths=None), dict(W=0), dict(W=sfc.MAX_PACKED_WIDTH + 1), dict(flags=1)]
GRAD_FAULTS = [dict(grad=None), dict(grad=FAR + 1), dict(grad_stride=15), dict(up=None),
               dict(grad=FAKE), dict(grad=FAKE + 64), dict(grad=FAKE - 64)]  # overlapping the logits


@pytest.mark.parametrize("fault", ROW_FAULTS + TEACHER_FAULTS + [dict(loss=None), dict(status=None), dict(stats=FAKE + 4)])
def test_distill_forward(lib, fault):
    a = {**ROWS, **TEACHER, "loss": FAKE, "stats": None, "status": FAKE, "stream": None, **fault}
    assert lib.sfc_distill_forward(*a.values()) == sfc.SFC_EINVAL


@pytest.mark.parametrize("fault", ROW_FAULTS + TEACHER_FAULTS + GRAD_FAULTS + [dict(stats=None), dict(stats=FAKE + 8)])
def test_distill_backward(lib, fault):
    a = {**ROWS, **TEACHER, "stats": FAKE, "up": FAKE, "grad": FAR, "grad_stride": 16, "stream": None, **fault}
    assert lib.sfc_distill_backward(*a.values()) == sfc.SFC_EINVAL


@pytest.mark.parametrize("fault", ROW_FAULTS + TEACHER_FAULTS + GRAD_FAULTS + [dict(loss=None), dict(status=None)])
def test_distill_forward_backward(lib, fault):
    a = {**ROWS, **TEACHER, "up": FAKE, "loss": FAKE, "status": FAKE, "grad": FAR, "grad_stride": 16, "stream": None, **fault}
    assert lib.sfc_distill_forward_backward(*a.values()) == sfc.SFC_EINVAL


@pytest.mark.parametrize("fault", ROW_FAULTS + GRAD_FAULTS + [dict(ids=None), dict(lengths=None), dict(W=0), dict(tokens=None),
                                                              dict(W=sfc.MAX_PACKED_WIDTH + 1)])
def test_replay_backward(lib, fault):
    a = {**ROWS, "ids": FAKE, "lengths": FAKE, "W": 8, "tokens": FAKE, "up": FAKE, "entries": None, "grad": FAR, "grad_stride": 16,
         "stream": None, **fault}
    assert lib.sfc_replay_backward(*a.values()) == sfc.SFC_EINVAL


VERIFY = dict(target=FAKE, draft=FAKE, dtype=0, B=3, D=2, V=16, treq=48, trow=16, dreq=32, drow=16, T=FAKE, Td=None, drafted=FAKE,
              n=None, u=FAKE, seed=0, step=0, row_offset=0, flags=0, acc=FAKE, tok=FAKE, lps=FAKE, status=FAKE, ws=FAKE,
              ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("fault", [dict(target=None), dict(dtype=2), dict(B=0), dict(D=0), dict(D=sfc.MAX_DRAFTS + 1), dict(V=0),
                                   dict(treq=-1), dict(trow=-1), dict(dreq=-1), dict(drow=-1), dict(T=None), dict(drafted=None),
                                   dict(u=None), dict(row_offset=-1), dict(row_offset=2 ** 32 - 2), dict(flags=2), dict(acc=None),
                                   dict(tok=None), dict(lps=None), dict(status=None), dict(target=FAKE + 1), dict(draft=FAKE + 1),
                                   dict(ws=FAKE + 8), dict(B=2 ** 31)])
def test_verify_drafts(lib, fault):
    assert lib.sfc_verify_drafts(*{**VERIFY, **fault}.values()) == sfc.SFC_EINVAL


def test_verify_drafts_workspace(lib):
    need = sfc.verify_workspace_size(3, 2, 16, sfc.SFC_BF16)
    assert need > 0 and sfc.verify_workspace_size(0, 2, 16, 0) == 0 and sfc.verify_workspace_size(3, 65, 16, 0) == 0
    assert lib.sfc_verify_drafts(*{**VERIFY, "ws": None}.values()) == sfc.SFC_EWORKSPACE
    assert lib.sfc_verify_drafts(*{**VERIFY, "ws_bytes": need - 1}.values()) == sfc.SFC_EWORKSPACE


@pytest.mark.parametrize("fault", [dict(tids=None), dict(tlps=None), dict(tlen=None), dict(tw=0), dict(tw=sfc.MAX_PACKED_WIDTH + 1),
                                   dict(dlps=None), dict(dlen=None), dict(dw=0), dict(dw=sfc.MAX_PACKED_WIDTH + 1), dict(B=0),
                                   dict(D=0), dict(D=sfc.MAX_DRAFTS + 1), dict(drafted=None), dict(u=None), dict(row_offset=-1),
                                   dict(row_offset=2 ** 32 - 2), dict(acc=None), dict(tok=None), dict(lps=None), dict(status=None)])
def test_verify_supports(lib, fault):
    a = dict(tids=FAKE, tlps=FAKE, tlen=FAKE, tw=8, dids=FAKE, dlps=FAKE, dlen=FAKE, dw=8, B=3, D=2, drafted=FAKE, n=None, u=FAKE,
             seed=0, step=0, row_offset=0, acc=FAKE, tok=FAKE, lps=FAKE, status=FAKE, stream=None)
    assert lib.sfc_verify_supports(*{**a, **fault}.values()) == sfc.SFC_EINVAL


def test_constants_match_the_header():
    import re

    src = open(os.path.join(os.path.dirname(__file__), "..", "include", "sfc.h")).read()
    consts = dict(re.findall(r"#define (SFC_[A-Z_0-9]+) \(?(-?\d+)u?\)?", src))
    assert int(consts["SFC_FLAG_NORMALISE_TEACHER"]) == sfc.FLAG_NORMALISE_TEACHER
    assert int(consts["SFC_MAX_DRAFTS"]) == sfc.MAX_DRAFTS


def test_row_layouts():
    f = training.check_row_layout
    assert f("x", torch.zeros(3, 10)) == 10
    assert f("x", torch.zeros(3, 16)[:, :10]) == 16
    assert f("x", torch.zeros(10).expand(1, 10)) == 10
    for bad in (torch.zeros(10), torch.zeros(0, 4), torch.zeros(3, 10, dtype=torch.float16), torch.zeros(10, 3).t(),
                torch.zeros(10).expand(3, 10), torch.zeros(3, 20)[:, ::2]):
        with pytest.raises(sfc.SfcError):
            f("x", bad)
    with pytest.raises(sfc.SfcError, match="CUDA"):
        training.check_rows("x", torch.zeros(3, 10))


def test_packed_layouts():
    x, T = torch.zeros(3, 10), torch.ones(3)
    ids, y, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4), torch.ones(3, dtype=torch.int32)
    assert training.check_packed(x, T, ids, n, y) == (x.device, 3, 4)
    for kw in (dict(ids=ids.long()), dict(ids=ids[:2]), dict(ids=ids.t().contiguous().t()), dict(ids=ids[:, :0]), dict(y=y.double()),
               dict(y=y[:, :3]), dict(n=n[:2]), dict(n=n.long()), dict(T=T[:2]), dict(T=T.double()),
               dict(ids=torch.zeros(3, sfc.MAX_PACKED_WIDTH + 1, dtype=torch.int32))):
        a = {"T": T, "ids": ids, "n": n, "y": y, **kw}
        with pytest.raises(sfc.SfcError):
            training.check_packed(x, a["T"], a["ids"], a["n"], a["y"])


def test_verify_layouts():
    B, D, V = 3, 2, 10
    base = dict(target=torch.zeros(B, D + 1, V), draft=torch.zeros(B, D, V), drafted=torch.zeros(B, D, dtype=torch.int32),
                u=torch.zeros(B, D), T=torch.ones(B), Td=None, n=None)
    f = lambda **kw: speculative.check_verify_layout(*{**base, **kw}.values())
    assert f() == (B, D, V, [30, 10, 20, 10])
    assert f(draft=None) == (B, D, V, [30, 10, 0, 0])
    assert f(target=torch.zeros(B, D + 1, 16)[:, :, :V])[3][:2] == [48, 16]
    assert f(target=torch.zeros(D + 1, B, V).transpose(0, 1))[3][:2] == [10, 30]  # position-major
    assert f(target=torch.zeros(D + 1, V).expand(B, D + 1, V))[3][:2] == [0, 10]
    for kw in (dict(target=torch.zeros(B, D, V)), dict(target=torch.zeros(B, D + 1, V + 1)), dict(draft=torch.zeros(B, D + 1, V)),
               dict(draft=torch.zeros(B, D, V, dtype=torch.bfloat16)), dict(target=torch.zeros(B, V, D + 1).transpose(1, 2)),
               dict(drafted=torch.zeros(B, D, dtype=torch.int64)),
               dict(drafted=torch.zeros(B, 0, dtype=torch.int32)), dict(u=torch.zeros(B, D + 1)), dict(T=torch.ones(B - 1)), dict(T=None),
               dict(Td=torch.ones(B, dtype=torch.float64)), dict(n=torch.zeros(B - 1, dtype=torch.int32))):
        with pytest.raises(sfc.SfcError):
            f(**kw)


def test_verify_supports_layouts():
    B, D = 3, 2
    i32 = torch.int32
    base = dict(tids=torch.zeros(B, D + 1, 5, dtype=i32), tlps=torch.zeros(B, D + 1, 5), tlen=torch.ones(B, D + 1, dtype=i32),
                dids=torch.zeros(B, D, 4, dtype=i32), dlps=torch.zeros(B, D, 4), dlen=torch.ones(B, D, dtype=i32),
                drafted=torch.zeros(B, D, dtype=i32), u=torch.zeros(B, D), n=None)
    f = lambda **kw: speculative.check_supports_layout(*{**base, **kw}.values())
    assert f() == (B, D, 5, 4) and f(dids=None, dlps=None, dlen=None) == (B, D, 5, 0)
    for kw in (dict(tids=torch.zeros(B, D, 5, dtype=i32)), dict(tlps=torch.zeros(B, D + 1, 4)), dict(tlen=torch.ones(B, D, dtype=i32)),
               dict(dlps=None), dict(dlen=None), dict(dids=torch.zeros(B, D, 4)), dict(tids=torch.zeros(B, D + 1, 0, dtype=i32)),
               dict(drafted=torch.zeros(B, 65, dtype=i32)), dict(n=torch.zeros(B))):
        with pytest.raises(sfc.SfcError):
            f(**kw)
