"""GPU parity of the policy loss and its gradient against the float64 oracle.

Tolerances as in test_token_logprobs_gpu. The ratio is exp(lp - old): off by the log-probability's half steps (of which the
division's remainder takes z's own), four of the exponential and those of the subtraction; the loss and the gradient's
slope are the ratio's multiples. Ratios keep 10^-3 from the range's borders, where the side is a matter of rounding.
"""
import numpy as np
import pytest

import oracle
from top_support_capture_gb300 import workloads as wl
from test_distill_gpu import HALF, _cuda, as_input, cuda, dev_logits  # noqa: F401 (the fixture)
from test_token_logprobs_gpu import close, grad_limit

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
LOW, HIGH = 0.2, 0.28


def make(B, V, dtype, seed, clipped=True, weight=0.0, spread=3.0):
    rng = np.random.default_rng(seed)
    l = as_input((rng.standard_normal((B, V)) * spread).astype(np.float32), dtype)
    T = rng.uniform(0.5, 1.7, B).astype(np.float32)
    tokens = rng.integers(0, V, B).astype(np.int32)
    c = dict(l=l, dtype=dtype, T=T, tokens=tokens, A=rng.standard_normal(B).astype(np.float32), g=rng.standard_normal(B).astype(np.float32),
             weight=weight, old=None)
    if clipped:
        shift = rng.choice([0.0, 0.1, -0.1, 0.5, -0.5], B) + rng.uniform(-0.01, 0.01, B)
        lp = oracle.token_logprobs(l, dtype, T, tokens).logprobs[:, 0]
        c["old"] = (lp - shift).astype(np.float32)
    if B > 3:
        c["tokens"][2] = -1
    return c


def reference(c):
    return oracle.policy_loss(c["l"], c["dtype"], c["T"], c["tokens"], c["A"], c["g"], c["old"], LOW, HIGH, c["weight"])


def call(c, grad=None, layout={}, **kw):
    import top_support_capture_gb300 as sfc

    old = None if c["old"] is None else cuda(c["old"], np.float32)
    return sfc.policy_loss_and_grad(dev_logits(c["l"], c["dtype"], **layout), cuda(c["T"], np.float32), cuda(c["tokens"], np.int32),
                                    cuda(c["A"], np.float32), cuda(c["g"], np.float32), old_logprobs=old, clip_low=LOW, clip_high=HIGH,
                                    entropy_weight=c["weight"], grad=grad, **kw)


def check(c, out):
    ref = reference(c)
    stats = oracle.token_logprobs(c["l"], c["dtype"], c["T"], np.where(ref.row_status == 0, c["tokens"], -1))
    np.testing.assert_array_equal(out.row_status.cpu().numpy(), ref.row_status)
    H, lp = np.nan_to_num(ref.entropy), np.nan_to_num(np.abs(ref.logprobs), posinf=0)
    off_lp = 104 + 4 * H + 6 * stats.ln_mass + 5 * lp  # half steps
    off_H = 104 + 106 * H + stats.ln_mass + 4 * stats.spread
    close(out.logprobs, ref.logprobs, HALF * off_lp)
    close(out.entropy, ref.entropy, HALF * off_H)
    old = 0.0 if c["old"] is None else np.abs(np.nan_to_num(c["old"], neginf=0.0))
    off_rho = off_lp + 2 * old + 8
    with np.errstate(invalid="ignore"):
        loss = np.nan_to_num(np.abs(ref.loss), posinf=0)
        size = np.abs(ref.slope) * (off_rho if c["old"] is not None else off_lp)
        limit = HALF * (size + abs(c["weight"]) * (off_H + 2 * H) + 4 * loss)
    close(out.loss, ref.loss, limit)
    got = out.grad_logits.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    more = (off_rho if c["old"] is not None else 0.0 * lp)[:, None]
    over = np.abs(got - ref.grad) - grad_limit(c, stats.far, ref.grad, ref.grad_scale, more)
    assert over.max() <= 0, (np.unravel_index(over.argmax(), over.shape), over.max())
    return ref


SHAPES = [(1, 1), (2, 7), (3, 8), (4, 31), (5, 1000), (4, 1024), (3, 4099), (3, 50021), (2, 151936), (2, 129280), (2, 262144), (1, 300001),
          (1, 900001), (40, 12345), (700, 257)]


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,V", SHAPES)
@pytest.mark.parametrize("clipped,weight", [(True, 0.0), (True, 0.05), (False, 0.0), (False, -0.3)])
def test_policy(dtype, B, V, clipped, weight):
    c = make(B, V, dtype, V, clipped, weight)
    check(c, call(c))


# by 16-byte vectors a row: what CTAs of each size hold at most and just above it, and rows over clusters
@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,vectors", [(320, 1656), (320, 1657), (320, 3320), (320, 3321), (310, 4429), (310, 4430), (200, 7500), (120, 18992),
                                       (60, 45000)])
def test_many_rows(dtype, B, vectors):
    V = vectors * (8 if dtype == wl.DT_BF16 else 4) + 3
    c = make(B, V, dtype, B + vectors, True, 0.01)
    out = call(c)
    assert not out.row_status.any() and torch.isfinite(out.loss).all()
    rows = np.unique(np.r_[0, 1, 2, B - 1, np.random.default_rng(B).integers(0, B, 5)])
    some = {**c, **{k: c[k][rows] for k in ("l", "T", "tokens", "A", "g", "old")}}
    at = torch.from_numpy(rows).cuda()
    check(some, type(out)(*(t[at] for t in out)))
    padded = torch.from_numpy(c["tokens"] < 0).cuda()
    assert not out.grad_logits[padded].any() and out.grad_logits[~padded].any(1).sum() > B // 2


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,V", [(5, 5003), (3, 100003), (320, 20001)])
@pytest.mark.parametrize("pad,offset,out_offset", [(1, 0, 0), (8, 8, 8), (3, 1, 1), (5, 0, 3), (16, 2, 0)])
def test_strides_and_alignments(dtype, B, V, pad, offset, out_offset):
    c = make(B, V, dtype, pad + offset, True, 0.1)
    buf = torch.full((B * (V + pad) + out_offset,), 7.0, dtype=torch.bfloat16 if dtype == wl.DT_BF16 else torch.float32, device="cuda")
    check(c, call(c, grad=buf[out_offset:].view(B, V + pad)[:, :V], layout=dict(pad=pad, offset=offset)))
    assert (buf[:out_offset] == 7).all() and (buf[out_offset:].view(B, V + pad)[:, V:] == 7).all()


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("clipped", [True, False])
def test_masked_extreme_and_bad_rows(dtype, clipped):
    B, V = 18, 2053
    c = make(B, V, dtype, 1, clipped, 0.02)
    l = oracle.widen_logits(c["l"], dtype).astype(np.float32)
    c["tokens"][:] = 100
    c["A"][:] = np.where(np.arange(B) % 2, -1.5, 0.75)
    c["T"][:] = 1.0
    if clipped:
        lp = oracle.token_logprobs(c["l"], dtype, c["T"], c["tokens"]).logprobs[:, 0]
        c["old"] = (lp - 0.05).astype(np.float32)
    l[0, 300:] = -np.inf
    l[1, 300:] = -3.3895313892515355e38
    l[2, :] = -3.3895313892515355e38
    l[3, :] = -np.inf
    l[4, 2000] = np.nan
    l[5, 7] = np.inf
    l[6, 100] = -np.inf  # the token
    l[7, 100] = -np.inf
    c["tokens"][8] = V
    c["tokens"][9] = -2
    c["tokens"][10] = -1
    l[10, :] = np.nan  # padding: its logits do not matter
    c["A"][11] = np.inf
    c["T"][12:15] = [0, np.inf, np.nan]
    c["A"][15] = 0.0
    c["tokens"][16] = -1
    c["T"][16] = -1.0  # bad all the same
    if clipped:
        c["old"][17] = -np.inf
        with np.errstate(over="ignore"):
            c["old"][0:3] = oracle.token_logprobs(as_input(l, dtype), dtype, c["T"], c["tokens"]).logprobs[0:3, 0] + 0.03
    c["l"] = as_input(l, dtype)
    ref = check(c, call(c))
    assert list(ref.row_status) == [0, 0, 0, -1, -1, -1, 0, 0, -1, -1, 0, -1, -1, -1, -1, 0, -1, -1 if clipped else 0]
    assert ref.slope[6] == 0 and ref.slope[7] == 0 and (clipped or (ref.loss[6] == np.inf and ref.loss[7] == -np.inf))


@pytest.mark.parametrize("B", [4, 320])
@pytest.mark.parametrize("shift", [-3e4, 1e6])
def test_shifted_logits(B, shift):
    """A constant added to a row changes nothing: the exponents' reference is far from 0 there."""
    c = make(B, 5003, wl.DT_F32, 13, False, 0.02)
    c["l"] = (c["l"] + np.float32(shift)).astype(np.float32)
    check(c, call(c))


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_masks_in_some_vectors_only(dtype):
    """Threads whose logits are all near beside threads with masked ones, and scales that are far from 1."""
    c = make(6, 30011, dtype, 14, False, 0.02)
    l = oracle.widen_logits(c["l"], dtype).astype(np.float32)
    l[0, 1000:1400] = -np.inf
    l[1, 7::513] = -3.3895313892515355e38
    l[2, 29000:] = -np.inf
    l[3] *= 1e4
    l[4] *= 1e-6
    c["T"][5] = 1e-30
    c["l"] = as_input(l, dtype)
    check(c, call(c))


def test_ratios_that_overflow():
    """An unclipped ratio above float32's range: an infinite loss, a gradient that stays a number."""
    c = make(2, 100, wl.DT_F32, 3)
    c["A"][:] = [-1.0, 1.0]
    c["old"][:] = -1000.0
    out = call(c)
    assert out.loss[0] == np.inf and not torch.isnan(out.grad_logits).any() and out.row_status.tolist() == [0, 0]
    assert float(out.loss[1]) == -np.float32(np.float32(1) + np.float32(HIGH)) and not out.grad_logits[1].any()


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("V", [3001, 129280])
def test_a_copy_that_never_arrives(dtype, V):
    c = make(6, V, dtype, 8)
    c["A"][4] = np.nan
    out = call(c, test_stall=True)
    assert out.row_status.tolist() == [-2, -2, 0, -2, -1, -2]
    assert torch.isnan(out.loss).tolist() == [True, True, False, True, True, True] and not out.grad_logits.any()
    check(c, call(c))


def test_the_same_as_autograd_over_token_logprobs():
    """The loss written with token_logprobs and elementary operations, and its gradient."""
    import top_support_capture_gb300 as sfc

    c = make(9, 30000, wl.DT_F32, 11, True, 0.03)
    c["tokens"][2] = 5
    out = call(c)
    x = dev_logits(c["l"], c["dtype"]).requires_grad_()
    o = sfc.token_logprobs(x, cuda(c["T"], np.float32), cuda(c["tokens"], np.int32))
    A, old = cuda(c["A"], np.float32), cuda(c["old"], np.float32)
    rho = (o.logprobs - old).exp()
    loss = -torch.minimum(rho * A, rho.clamp(1 - LOW, 1 + HIGH) * A) - c["weight"] * o.entropy
    (grad,) = torch.autograd.grad(loss, x, cuda(c["g"], np.float32))
    ref = check(c, out)
    check(c, type(out)(loss.detach(), o.logprobs.detach(), o.entropy.detach(), grad, o.row_status))
    assert np.count_nonzero(ref.slope) not in (0, 9)  # some clipped, some not


def test_streams_graphs_and_repeats():
    import top_support_capture_gb300 as sfc

    c = make(6, 40960, wl.DT_BF16, 9, True, 0.01)
    first = call(c)
    again = call(c)
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    x, T, t, A, g, old = (dev_logits(c["l"], c["dtype"]), cuda(c["T"], np.float32), cuda(c["tokens"], np.int32), cuda(c["A"], np.float32),
                          cuda(c["g"], np.float32), cuda(c["old"], np.float32))
    run = lambda **kw: sfc.policy_loss_and_grad(x, T, t, A, g, old_logprobs=old, clip_low=LOW, clip_high=HIGH, entropy_weight=0.01, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    A.mul_(-1.0)
    c["A"] = -c["A"]
    graph.replay()
    torch.cuda.synchronize()
    check(c, held)


def test_rows_past_32_bit_offsets():
    import top_support_capture_gb300 as sfc

    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    V, B, last = 262144, 8200, 2
    c = make(last, V, wl.DT_BF16, 5, True, 0.01)
    big = torch.empty((B, V), dtype=torch.bfloat16, device="cuda")
    big[-last:] = dev_logits(c["l"], c["dtype"])
    full = lambda v, dt: torch.full((B,), v, dtype=dt, device="cuda")
    T, t, A, g, old = full(1, torch.float32), full(-1, torch.int32), full(1, torch.float32), full(1, torch.float32), full(0, torch.float32)
    for whole, part in ((T, "T"), (t, "tokens"), (A, "A"), (g, "g"), (old, "old")):
        whole[-last:] = torch.from_numpy(c[part]).cuda()
    grad = torch.full((B, V), 3.0, dtype=torch.bfloat16, device="cuda")
    out = sfc.policy_loss_and_grad(big, T, t, A, g, old_logprobs=old, clip_low=LOW, clip_high=HIGH, entropy_weight=0.01, grad=grad)
    check(c, type(out)(*(v[-last:] for v in out)))
    assert not out.loss[:-last].any() and not grad[:-last].any()
