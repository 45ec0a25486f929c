"""GPU parity of the distillation loss and gradient and of the replay's gradient against the float64 oracle.

Tolerances, counted from the roundings before the first run. A loss is a sum of terms t (ln t - z): t is within
2^-22 (expf, its product), z within 3 half steps, the sum of at most 16384 entries in 512 shares of 32 within
(32 + 21) half steps, and ln of the row's mass within 2^-22 + 4 |z| half steps of the exponents; together under
128 half steps (2^-17) of the terms' magnitudes. A gradient entry is a difference of k p and t g / T: p is within
(64 + 8 |z - z_max|) half steps (three roundings of the exponent, times ln 2 each, the mass, k), and the result is
rounded once to the output's type. Results below the smallest normal number may be flushed.
"""
import numpy as np
import pytest

import oracle
from top_support_capture_gb300 import workloads as wl

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import top_support_capture_gb300 as sfc

    sfc.load_library()


def dev_logits(x, dtype, pad=0, offset=0):
    """The logits on the GPU, in rows V + pad apart that start `offset` elements into their buffer."""
    x = np.ascontiguousarray(x)
    t = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16) if dtype == wl.DT_BF16 else torch.from_numpy(x).cuda()
    if not pad and not offset:
        return t
    B, V = t.shape
    buf = torch.full((B * (V + pad) + offset,), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[offset:].view(B, V + pad)[:, :V]
    view.copy_(t)
    return view


def as_input(l, dtype):
    return wl.f32_to_bf16_bits(l) if dtype == wl.DT_BF16 else l.astype(np.float32)


def cuda(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a, dt)).cuda()


def make(B, V, W, dtype, seed, normalise=False, spread=3.0):
    rng = np.random.default_rng(seed)
    l = as_input((rng.standard_normal((B, V)) * spread).astype(np.float32), dtype)
    k = min(W, V)
    ids = np.full((B, W), -1, np.int32)
    y = np.full((B, W), np.nan, np.float32)  # past the length: never read
    lens = rng.integers(0, k + 1, size=B).astype(np.int32)
    lens[:3] = [k, 0, 1][:min(3, B)]
    for r in range(B):
        n = lens[r]
        ids[r, :n] = rng.choice(V, n, replace=False)
        v = rng.standard_normal(n).astype(np.float32) * 2
        y[r, :n] = v if normalise or n == 0 else v - np.log(np.exp(v.astype(np.float64)).sum()).astype(np.float32)
    T = rng.uniform(0.5, 1.7, B).astype(np.float32)
    g = rng.standard_normal(B).astype(np.float32)
    return dict(l=l, dtype=dtype, T=T, ids=ids, y=y, lens=lens, W=W, g=g, normalise=normalise)


def reference(c):
    return oracle.distill(c["l"], c["dtype"], c["T"], c["ids"], c["y"], c["lens"], c["W"], c["g"], c["normalise"])


def args(c, **layout):
    return (dev_logits(c["l"], c["dtype"], **layout), cuda(c["T"], np.float32), cuda(c["ids"], np.int32),
            cuda(c["y"], np.float32), cuda(c["lens"], np.int32))


def check_loss(ref, loss, status):
    np.testing.assert_array_equal(status.cpu().numpy(), ref.row_status)
    loss = loss.cpu().numpy().astype(np.float64)
    fine = np.isfinite(ref.loss)
    np.testing.assert_array_equal(loss[~fine], ref.loss[~fine])  # NaN and inf where the oracle has them
    assert np.all(np.abs(loss - ref.loss)[fine] <= 128 * HALF * (1 + ref.loss_scale[fine]))


def grad_limit(c, want, scale):
    z = oracle.widen_logits(c["l"], c["dtype"]) / c["T"].astype(np.float64)[:, None]
    with np.errstate(invalid="ignore"):
        far = np.nan_to_num(np.abs(z - np.nanmax(np.where(np.isfinite(z), z, np.nan), axis=1, keepdims=True)), nan=0, posinf=0)
    step = 2.0 ** -9 * 2 if c["dtype"] == wl.DT_BF16 else HALF
    return step * np.abs(want) + (64 + 8 * np.minimum(far, 100)) * HALF * scale * (1 + step) + 2.0 ** -126


def check_grad(c, ref, grad):
    got = grad.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    over = np.abs(got - ref.grad) - grad_limit(c, ref.grad, ref.grad_scale)
    assert over.max() <= 0, (np.unravel_index(over.argmax(), over.shape), over.max())


SHAPES = [(1, 1, 1), (2, 7, 3), (3, 8, 8), (4, 31, 64), (5, 1000, 1), (4, 1024, 1024), (3, 4099, 33), (3, 50021, 1024),
          (2, 151936, 1024), (2, 129280, 8192), (2, 262144, 16384), (1, 300001, 7), (1, 900001, 2000), (40, 12345, 600), (700, 257, 40)]


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,V,W", SHAPES)
@pytest.mark.parametrize("normalise", [False, True])
def test_distill(dtype, B, V, W, normalise):
    import top_support_capture_gb300 as sfc

    c = make(B, V, W, dtype, V + W, normalise)
    ref, a = reference(c), args(c)
    out = sfc.distill_loss_and_grad(*a, cuda(c["g"], np.float32), normalise=normalise)
    check_loss(ref, out.loss, out.row_status)
    check_grad(c, ref, out.grad_logits)
    # the loss alone, and the gradient through autograd
    x = a[0].detach().requires_grad_()
    two = sfc.distill_loss(x, *a[1:], normalise=normalise)
    check_loss(ref, two.loss.detach(), two.row_status)
    (grad,) = torch.autograd.grad(two.loss, x, cuda(c["g"], np.float32))
    check_grad(c, ref, grad)
    alone = sfc.distill_loss(*a, normalise=normalise)
    assert alone.loss.grad_fn is None
    check_loss(ref, alone.loss, alone.row_status)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("pad,offset,out_offset", [(1, 0, 0), (8, 8, 8), (3, 1, 1), (5, 0, 3), (16, 2, 0)])
def test_strides_and_alignments(dtype, pad, offset, out_offset):
    """Rows apart, starting anywhere, and a gradient that lies differently from its logits; nothing around the
    gradient's rows is written."""
    import top_support_capture_gb300 as sfc

    B, V = 5, 5003
    c = make(B, V, 100, dtype, pad + offset)
    ref, a = reference(c), args(c, pad=pad, offset=offset)
    buf = torch.full((B * (V + pad) + out_offset,), 7.0, dtype=a[0].dtype, device="cuda")
    grad = buf[out_offset:].view(B, V + pad)[:, :V]
    out = sfc.distill_loss_and_grad(*a, cuda(c["g"], np.float32), grad=grad)
    check_loss(ref, out.loss, out.row_status)
    check_grad(c, ref, grad)
    assert (buf[:out_offset] == 7).all() and (buf[out_offset:].view(B, V + pad)[:, V:] == 7).all()
    x = a[0].detach().requires_grad_()
    (grad,) = torch.autograd.grad(sfc.distill_loss(x, *a[1:]).loss, x, cuda(c["g"], np.float32))
    check_grad(c, ref, grad)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_masked_and_extreme_logits(dtype):
    """-inf and lowest values, rows without a finite logit, NaN, +inf; teachers with empty, -inf and bad entries."""
    import top_support_capture_gb300 as sfc

    B, V, W = 14, 2053, 6
    c = make(B, V, W, dtype, 1)
    l = oracle.widen_logits(c["l"], dtype).astype(np.float32)
    low = np.float32(-3.3895313892515355e38)  # bfloat16's lowest value
    c["lens"][:] = W
    rng = np.random.default_rng(0)
    for r in range(B):
        c["ids"][r] = rng.choice(np.arange(100, 200), W, replace=False)
        c["y"][r] = np.log(np.float32(1 / W))
    l[0, 300:] = -np.inf
    l[1, 300:] = low
    l[2, :] = low
    l[3, :] = -np.inf
    l[4, 2000] = np.nan
    l[5, 7] = np.inf
    l[6, c["ids"][6, 2]] = -np.inf  # the student gives a teacher's token no probability: an infinite loss
    c["y"][7, 3] = -np.inf
    c["y"][8, 1] = np.nan
    c["y"][9, 0] = np.inf
    c["ids"][10, 5] = V
    c["ids"][11, 0] = -1
    c["lens"][12] = W + 3  # the first W entries are the teacher
    c["lens"][13] = -1
    c["l"] = as_input(l, dtype)
    for normalise in (False, True):
        c["normalise"] = normalise
        ref = reference(c)
        assert list(ref.row_status) == [0, 0, 0, -1, -1, -1, 0, 0, -1, -1, -1, -1, 1, -1]
        assert ref.loss[6] == np.inf
        out = sfc.distill_loss_and_grad(*args(c), cuda(c["g"], np.float32), normalise=normalise)
        check_loss(ref, out.loss, out.row_status)
        check_grad(c, ref, out.grad_logits)
        x = args(c)[0].requires_grad_()
        loss = sfc.distill_loss(x, *args(c)[1:], normalise=normalise).loss
        (grad,) = torch.autograd.grad(loss, x, cuda(c["g"], np.float32))
        check_grad(c, ref, grad)


def test_bad_temperatures():
    import top_support_capture_gb300 as sfc

    c = make(6, 100, 4, wl.DT_F32, 2)
    c["lens"][:] = 2
    c["ids"][:, :2], c["y"][:, :2] = [3, 4], np.log(0.5)
    c["T"][:] = [0, -1, np.inf, np.nan, 1e-3, 1e4]
    ref = reference(c)
    assert list(ref.row_status) == [-1, -1, -1, -1, 0, 0]
    out = sfc.distill_loss_and_grad(*args(c), cuda(c["g"], np.float32))
    np.testing.assert_array_equal(out.row_status.cpu().numpy(), ref.row_status)
    assert torch.isnan(out.loss[:4]).all() and (out.grad_logits[:4] == 0).all()
    np.testing.assert_allclose(out.loss[4:].cpu().numpy(), ref.loss[4:], rtol=128 * HALF)


def test_reductions_and_training_step():
    """loss.mean().backward() (an expanded upstream gradient), repeated calls giving the same bits, and the
    captured training step."""
    import top_support_capture_gb300 as sfc

    c = make(6, 4096, 32, wl.DT_BF16, 9)
    a = args(c)
    x = a[0].detach().requires_grad_()
    sfc.distill_loss(x, *a[1:]).loss.mean().backward()
    c["g"] = np.full(6, 1 / 6, np.float32)
    ref = reference(c)
    check_grad(c, ref, x.grad)
    g = cuda(c["g"], np.float32)
    first = sfc.distill_loss_and_grad(*a, g)
    again = sfc.distill_loss_and_grad(*a, g)
    assert torch.equal(first.loss, again.loss) and torch.equal(first.grad_logits, again.grad_logits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sfc.distill_loss_and_grad(*a, g, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first.grad_logits, other.grad_logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = sfc.distill_loss_and_grad(*a, g)
    a[0].add_(1.0)  # new inputs in the same place (adding 1 to every logit changes no softmax beyond rounding)
    graph.replay()
    torch.cuda.synchronize()
    c["l"] = a[0].view(torch.int16).cpu().numpy().view(np.uint16)
    check_loss(reference(c), held.loss, held.row_status)
    check_grad(c, reference(c), held.grad_logits)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("V", [3001, 129280])
def test_a_copy_that_never_arrives(dtype, V):
    """The bounded wait for a kept slice gives up: every row that has work reports the timeout, with a NaN loss and
    no gradient; rows without a teacher and bad rows are as ever; and the next call is right."""
    import top_support_capture_gb300 as sfc

    c = make(6, V, 16, dtype, 8)
    c["lens"][:] = [16, 0, 3, 16, -1, 2]
    for r, n in ((0, 16), (2, 3), (3, 16), (5, 2)):
        c["ids"][r, :n], c["y"][r, :n] = np.arange(n), np.log(1 / n)
    a, g = args(c), cuda(c["g"], np.float32)
    out = sfc.distill_loss_and_grad(*a, g, test_stall=True)
    assert list(out.row_status.cpu()) == [-2, 0, -2, -2, -1, -2]
    assert list(torch.isnan(out.loss).cpu()) == [True, False, True, True, True, True] and out.loss[1] == 0
    assert not out.grad_logits.any()
    ref, out = reference(c), sfc.distill_loss_and_grad(*a, g)
    check_loss(ref, out.loss, out.row_status)
    check_grad(c, ref, out.grad_logits)


# ------------------------------------------------------------------------------------------------ replay


def replay_case(B, V, W, dtype, seed):
    c = make(B, V, W, dtype, seed)
    rng = np.random.default_rng(seed + 1)
    c["lens"] = np.maximum(c["lens"], 1).astype(np.int32)
    for r in range(B):
        c["ids"][r, :c["lens"][r]] = rng.choice(V, c["lens"][r], replace=False)
    c["tok"] = np.array([c["ids"][r, rng.integers(c["lens"][r])] for r in range(B)], np.int32)
    c["G"] = rng.standard_normal((B, W)).astype(np.float32)
    return c


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,V,W", SHAPES)
def test_replay_gradient(dtype, B, V, W):
    import top_support_capture_gb300 as sfc

    c = replay_case(B, V, W, dtype, V)
    a = (dev_logits(c["l"], dtype), cuda(c["T"], np.float32), cuda(c["ids"], np.int32), cuda(c["lens"], np.int32), cuda(c["tok"], np.int32))
    g, G = cuda(c["g"], np.float32), cuda(c["G"], np.float32)
    for entries in (None, "G"):
        grad, mag = oracle.replay_gradient(c["l"], dtype, c["T"], c["ids"], c["lens"], W, c["tok"], c["g"], c["G"] if entries else None)
        ref = oracle.DistillResult(None, grad, None, mag, None)
        check_grad(c, ref, sfc.replay_logprob_backward(*a, g, grad_support_logprobs=G if entries else None))
        x = a[0].detach().requires_grad_()
        out = sfc.replay_logprob(x, *a[1:], support_logprobs=bool(entries))
        plain = sfc.replay_logprob(*a, support_logprobs=bool(entries))
        assert torch.equal(out.token_logprob, plain.token_logprob)  # the same call, the same bits
        outs, ups = ([out.token_logprob, out.support_logprobs], [g, G]) if entries else ([out.token_logprob], [g])
        check_grad(c, ref, torch.autograd.grad(outs, x, ups)[0])


def test_replay_gradient_of_rows_without_a_logprob():
    import top_support_capture_gb300 as sfc

    V, W = 100, 8
    l = np.zeros((8, V), np.float32)
    l[:, :5] = [3.0, 2.0, 1.0, 0.0, -1.0]
    ids = np.tile(np.array([0, 1, 2, 3, -1, -1, -1, -1], np.int32), (8, 1))
    lens = np.array([4, 4, 9, 0, 4, 4, 4, 4], np.int32)
    toks = np.array([2, 50, 0, 0, 0, 0, 0, 1], np.int32)
    T = np.array([1, 1, 1, 1, 0, np.inf, 1, 1], np.float32)
    ids[6, 3] = V
    l[7, 1] = np.nan
    G = np.random.default_rng(0).standard_normal((8, W)).astype(np.float32)
    want, mag = oracle.replay_gradient(l, wl.DT_F32, T, ids, lens, W, toks, np.ones(8), G)
    assert np.abs(want[:2]).max() > 0 and (want[2:] == 0).all()
    got = sfc.replay_logprob_backward(dev_logits(l, wl.DT_F32), cuda(T, np.float32), cuda(ids, np.int32), cuda(lens, np.int32),
                                      cuda(toks, np.int32), torch.ones(8, device="cuda"), cuda(G, np.float32)).cpu().numpy()
    assert (got[2:] == 0).all()
    assert np.all(np.abs(got[:2] - want[:2]) <= HALF * np.abs(want[:2]) + 128 * HALF * mag[:2])


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("pad,out_offset", [(0, 1), (3, 0), (5, 3), (8, 8)])
def test_replay_gradient_writes_its_rows_only(dtype, pad, out_offset):
    import top_support_capture_gb300 as sfc

    B, V, W = 5, 5003, 64
    c = replay_case(B, V, W, dtype, 3)
    a = (dev_logits(c["l"], dtype, pad=pad), cuda(c["T"], np.float32), cuda(c["ids"], np.int32), cuda(c["lens"], np.int32),
         cuda(c["tok"], np.int32))
    buf = torch.full((B * (V + pad) + out_offset,), 7.0, dtype=a[0].dtype, device="cuda")
    grad = buf[out_offset:].view(B, V + pad)[:, :V]
    sfc.replay_logprob_backward(*a, cuda(c["g"], np.float32), grad=grad)
    want, mag = oracle.replay_gradient(c["l"], dtype, c["T"], c["ids"], c["lens"], W, c["tok"], c["g"])
    check_grad(c, oracle.DistillResult(None, want, None, mag, None), grad)
    assert (buf[:out_offset] == 7).all() and (buf[out_offset:].view(B, V + pad)[:, V:] == 7).all()


@pytest.mark.parametrize("dtype", [wl.DT_BF16])
def test_rows_past_32_bit_offsets(dtype):
    """Rows that start more than 2^31 elements (2^32 bytes) into their array; all others have no teacher."""
    import top_support_capture_gb300 as sfc

    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    V, B, W, last = 262144, 8200, 8, 2
    assert (B - last) * V > 2 ** 31
    c = make(last, V, W, dtype, 5)
    c["lens"][:] = W
    for r in range(last):
        c["ids"][r] = np.random.default_rng(r).choice(V, W, replace=False)
        c["y"][r] = np.log(1 / W)
    big = torch.empty((B, V), dtype=torch.bfloat16, device="cuda")
    big[-last:] = dev_logits(c["l"], dtype)
    T, g = torch.ones(B, device="cuda"), torch.zeros(B, device="cuda")
    T[-last:], g[-last:] = cuda(c["T"], np.float32), cuda(c["g"], np.float32)
    ids, y = torch.zeros((B, W), dtype=torch.int32, device="cuda"), torch.zeros((B, W), device="cuda")
    ids[-last:], y[-last:] = cuda(c["ids"], np.int32), cuda(c["y"], np.float32)
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    n[-last:] = W
    ref = reference(c)
    grad = torch.full((B, V), 3.0, dtype=torch.bfloat16, device="cuda")
    out = sfc.distill_loss_and_grad(big, T, ids, y, n, g, grad=grad)
    check_loss(ref, out.loss[-last:], out.row_status[-last:])
    check_grad(c, ref, grad[-last:])
    assert (out.loss[:-last] == 0).all() and not grad[:-last].any()
    x = big.requires_grad_()
    (grad,) = torch.autograd.grad(sfc.distill_loss(x, T, ids, y, n).loss, x, g)
    check_grad(c, ref, grad[-last:])
    del x
    tok = ids[:, 0].contiguous()
    want, mag = oracle.replay_gradient(c["l"], dtype, c["T"], c["ids"], c["lens"], W, c["ids"][:, 0], c["g"])
    got = sfc.replay_logprob_backward(big.detach(), T, ids, n, tok, g)
    check_grad(c, oracle.DistillResult(None, want, None, mag, None), got[-last:])
    assert not got[:-last].any()
