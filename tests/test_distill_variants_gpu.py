"""Every way that the distillation cuts its rows, against the oracle on some of them: many rows with a teacher in CTAs of
128, 256 and 384 threads (up to the longest rows of each and just past them), clusters that prefetch a later row's
slice, and gradients that lie differently from their logits across slices. Tolerances as in test_distill_gpu."""
import numpy as np
import pytest

from top_support_capture_gb300 import workloads as wl
from test_distill_gpu import _cuda, args, check_grad, check_loss, cuda, make, reference  # noqa: F401 (the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def rows_of(c, rows):
    return {**c, **{k: c[k][rows] for k in ("l", "T", "ids", "y", "lens", "g")}}


def check_some(c, out_loss, out_status, grad=None, count=10):
    """Statuses and finiteness of all rows; the first, last and some others against the oracle."""
    B = len(c["T"])
    assert not out_status.any() and torch.isfinite(out_loss).all()
    rows = np.unique(np.r_[0, 1, 2, B - 1, np.random.default_rng(B).integers(0, B, count)])
    some = rows_of(c, rows)
    ref, at = reference(some), torch.from_numpy(rows).cuda()
    check_loss(ref, out_loss[at], out_status[at])
    if grad is not None:
        empty = torch.from_numpy(c["lens"] == 0).cuda()
        assert torch.isfinite(grad).all() and not grad[empty].any() and grad[~empty].any(1).all()
        check_grad(some, ref, grad[at])


# by 16-byte vectors a row: CTAs of 128 up to 1656, of 256 up to 3320, of 384 up to 4429, then clusters of 512
VECTORS = [1656, 1657, 2500, 3320, 3321, 4000, 4429, 4430]


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("vectors", VECTORS)
@pytest.mark.parametrize("ragged,normalise", [(0, False), (3, True)])
def test_many_rows(dtype, vectors, ragged, normalise):
    import top_support_capture_gb300 as sfc

    V = vectors * (8 if dtype == wl.DT_BF16 else 4) + ragged
    c = make(320, V, 90, dtype, V, normalise)
    a, g = args(c), cuda(c["g"], np.float32)
    out = sfc.distill_loss_and_grad(*a, g, normalise=normalise)
    check_some(c, out.loss, out.row_status, out.grad_logits)
    x = a[0].detach().requires_grad_()
    two = sfc.distill_loss(x, *a[1:], normalise=normalise)
    (grad,) = torch.autograd.grad(two.loss, x, g)
    check_some(c, two.loss.detach(), two.row_status, grad)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,vectors", [(400, 6252), (200, 7500), (120, 18992), (60, 45000)])
def test_clusters_that_prefetch(dtype, B, vectors):
    """One, two, three and seven slices a row, more rows than a prefetch runs ahead."""
    import top_support_capture_gb300 as sfc

    V = vectors * (8 if dtype == wl.DT_BF16 else 4) + 5
    c = make(B, V, 700, dtype, B)
    out = sfc.distill_loss_and_grad(*args(c), cuda(c["g"], np.float32))
    check_some(c, out.loss, out.row_status, out.grad_logits, count=4)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,V,pad,offset,out_offset", [(5, 50021, 3, 1, 4), (5, 50024, 0, 0, 1), (40, 100003, 5, 2, 3), (320, 20001, 7, 3, 0),
                                                       (320, 30011, 0, 0, 5)])
def test_shifted_gradients_across_slices(dtype, B, V, pad, offset, out_offset):
    import top_support_capture_gb300 as sfc

    c = make(B, V, 200, dtype, V)
    a, g = args(c, pad=pad, offset=offset), cuda(c["g"], np.float32)
    buf = torch.full((B * (V + pad) + out_offset,), 7.0, dtype=a[0].dtype, device="cuda")
    grad = buf[out_offset:].view(B, V + pad)[:, :V]
    out = sfc.distill_loss_and_grad(*a, g, grad=grad)
    check_some(c, out.loss, out.row_status, grad)
    assert (buf[:out_offset] == 7).all() and (buf[out_offset:].view(B, V + pad)[:, V:] == 7).all()
    x = a[0].detach().requires_grad_()
    (grad,) = torch.autograd.grad(sfc.distill_loss(x, *a[1:]).loss, x, g)
    check_some(c, out.loss, out.row_status, grad)
