"""GPU parity of whole-vocabulary log-probabilities, entropies, top alternatives and their gradient against the float64 oracle.

Tolerances, counted from the roundings before the first run, in half steps (2^-24). A row's exponent d = (x - m) c has three
roundings and the exponential one of 2^-22: an exponential is within 4 + 4 |z - max z| of itself. The mass is a sum of
those over at most 512 shares, each of up to 300 terms in four lanes: with the sum's own (75 + 21), its logarithm is within
100 + 4 (their mean |z - max z|, at most the entropy). A log-probability adds three roundings of z - max z and the
sum's. The entropy's other part is sum e d / sum e: 100 + 4 mean + 4 spread, spread = sum p (z - max z)^2. Gradients: an
entry is a difference of g and p (G + h (ln p + H)), whose magnitudes the oracle adds up; p is within 100 + 8 |z - max z|,
G within as many half steps as tokens, and the result is rounded once to the output's type.
"""
import numpy as np
import pytest

import oracle
from top_support_capture_gb300 import workloads as wl
from test_distill_gpu import HALF, _cuda, as_input, cuda, dev_logits  # noqa: F401 (the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
LOW = np.float32(-3.3895313892515355e38)  # bfloat16's lowest value


def make(B, V, M, dtype, seed, spread=3.0):
    rng = np.random.default_rng(seed)
    l = as_input((rng.standard_normal((B, V)) * spread).astype(np.float32), dtype)
    tokens = rng.integers(-1, V, (B, M)).astype(np.int32)
    if M > 2:
        tokens[:, 2] = tokens[:, 0]  # the same token twice
    return dict(l=l, dtype=dtype, T=rng.uniform(0.5, 1.7, B).astype(np.float32), tokens=tokens,
                g=rng.standard_normal((B, M)).astype(np.float32), h=rng.standard_normal(B).astype(np.float32))


def reference(c, top=0):
    return oracle.token_logprobs(c["l"], c["dtype"], c["T"], c["tokens"], top)


def args(c, **layout):
    return dev_logits(c["l"], c["dtype"], **layout), cuda(c["T"], np.float32), cuda(c["tokens"], np.int32)


def close(got, want, limit):
    got = got.detach().cpu().numpy().astype(np.float64)
    want = np.where(np.abs(want) > np.finfo(np.float32).max * (1 + HALF / 2), np.copysign(np.inf, want), want)  # as float32 has it
    fine = np.isfinite(want)
    np.testing.assert_array_equal(got[~fine], want[~fine])  # NaN and -inf where the oracle has them
    over = np.abs(got - want)[fine] - np.broadcast_to(limit, want.shape)[fine]
    assert over.size == 0 or over.max() <= 0, over.max()


def check_values(c, ref, out, top=0):
    np.testing.assert_array_equal(out.row_status.cpu().numpy(), ref.row_status)
    H = np.nan_to_num(ref.entropy)
    mass = 104 + 4 * H + ref.ln_mass
    with np.errstate(invalid="ignore"):
        far = lambda lp: np.nan_to_num(np.abs(lp), posinf=0, neginf=0)
        if out.logprobs is not None:
            want = ref.logprobs.reshape(tuple(out.logprobs.shape))
            per = mass.reshape(-1, *[1] * (want.ndim - 1))
            close(out.logprobs, want, HALF * (per + 5 * far(want) + 5 * ref.ln_mass.reshape(per.shape)))
        close(out.entropy, ref.entropy, HALF * (mass + 102 * H + 4 * ref.spread))
        if top:
            np.testing.assert_array_equal(out.top_ids.cpu().numpy(), ref.top_ids)
            close(out.top_logprobs, ref.top_logprobs, HALF * (mass[:, None] + 5 * far(ref.top_logprobs) + 5 * ref.ln_mass[:, None]))
        else:
            assert out.top_ids is None and out.top_logprobs is None


def grad_limit(c, far, want, scale, more=0.0):
    """`more`: half steps of what the gradient's own factor is off by, per row."""
    step = 2.0 ** -8 if c["dtype"] == wl.DT_BF16 else HALF
    return step * np.abs(want) + (128 + more + 8 * np.minimum(far, 100)) * HALF * scale * (1 + step) + 2.0 ** -126


def check_grad(c, ref, want, grad):
    got = grad.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    over = np.abs(got - want.grad) - grad_limit(c, ref.far, want.grad, want.grad_scale)
    assert over.max() <= 0, (np.unravel_index(over.argmax(), over.shape), over.max())


SHAPES = [(1, 1, 1, 1), (2, 7, 3, 3), (3, 8, 1, 8), (4, 31, 5, 64), (5, 1000, 1, 20), (4, 1024, 2, 5), (3, 4099, 64, 64),
          (3, 50021, 4, 20), (1, 151936, 1, 20), (2, 129280, 8, 64), (2, 262144, 1, 1), (1, 300001, 7, 33), (40, 12345, 3, 10),
          (700, 257, 1, 5), (320, 4001, 2, 64), (160, 30011, 1, 2)]


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,V,M,top", SHAPES)
def test_token_logprobs(dtype, B, V, M, top):
    import top_support_capture_gb300 as sfc

    c = make(B, V, M, dtype, V + M)
    ref, a = reference(c, top), args(c)
    out = sfc.token_logprobs(*a, top=top)
    check_values(c, ref, out, top)
    # without alternatives, without tokens, as one token a row: the same bits
    bare = sfc.token_logprobs(*a)
    assert torch.equal(bare.logprobs, out.logprobs) and torch.equal(bare.entropy, out.entropy) and bare.top_ids is None
    none = sfc.token_logprobs(*a[:2], top=top)
    assert none.logprobs is None and torch.equal(none.entropy, out.entropy) and torch.equal(none.top_ids, out.top_ids)
    one = sfc.token_logprobs(*a[:2], a[2][:, 0].contiguous())
    assert one.logprobs.shape == (B,) and torch.equal(one.logprobs, out.logprobs[:, 0])
    # the gradient through autograd, and outside it
    want = oracle.token_logprobs_gradient(c["l"], dtype, c["T"], c["tokens"], c["g"], c["h"])
    g, h = cuda(c["g"], np.float32), cuda(c["h"], np.float32)
    x = a[0].detach().requires_grad_()
    two = sfc.token_logprobs(x, *a[1:], top=top)
    assert torch.equal(two.logprobs, out.logprobs) and not two.row_status.requires_grad
    (grad,) = torch.autograd.grad([two.logprobs, two.entropy], x, [g, h])
    check_grad(c, ref, want, grad)
    stats = sfc.token_logprobs(*a, keep_stats=True).row_stats
    assert torch.equal(sfc.token_logprobs_backward(*a, stats, g, h), grad)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_each_gradient_alone(dtype):
    """Of the log-probabilities, the entropy, the alternatives, and all together (tokens that are alternatives too)."""
    import top_support_capture_gb300 as sfc

    B, V, M, K = 4, 3001, 5, 64
    c = make(B, V, M, dtype, 2)
    ref, a = reference(c, K), args(c)
    c["tokens"][:, 1] = ref.top_ids[:, 3]
    a = args(c)
    ref = reference(c, K)
    gk = np.random.default_rng(1).standard_normal((B, K)).astype(np.float32)
    g, h, k = cuda(c["g"], np.float32), cuda(c["h"], np.float32), cuda(gk, np.float32)
    x = a[0].detach().requires_grad_()
    out = sfc.token_logprobs(x, *a[1:], top=K)
    both = np.concatenate([c["tokens"], ref.top_ids], 1)
    zero = np.zeros_like
    for outs, ups, parts in (([out.logprobs], [g], (c["g"], zero(gk), zero(c["h"]))), ([out.entropy], [h], (zero(c["g"]), zero(gk), c["h"])),
                             ([out.top_logprobs], [k], (zero(c["g"]), gk, zero(c["h"]))),
                             ([out.logprobs, out.top_logprobs, out.entropy], [g, k, h], (c["g"], gk, c["h"]))):
        want = oracle.token_logprobs_gradient(c["l"], dtype, c["T"], both, np.concatenate(parts[:2], 1), parts[2])
        check_grad(c, ref, want, torch.autograd.grad(outs, x, ups, retain_graph=True)[0])
    # an expanded upstream gradient; nothing of a loss that takes no output
    (-out.logprobs.mean()).backward()
    want = oracle.token_logprobs_gradient(c["l"], dtype, c["T"], c["tokens"], np.full((B, M), -1 / (B * M), np.float32))
    check_grad(c, ref, want, x.grad)
    # the entropy alone of a call without tokens
    y = a[0].detach().requires_grad_()
    (grad,) = torch.autograd.grad(sfc.token_logprobs(y, a[1]).entropy, y, h)
    check_grad(c, ref, oracle.token_logprobs_gradient(c["l"], dtype, c["T"], c["tokens"], zero(c["g"]), c["h"]), grad)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_gradient_against_differences(dtype):
    """Differences of the call's own values along a random direction."""
    import top_support_capture_gb300 as sfc

    B, V, M = 3, 500, 2
    c = make(B, V, M, wl.DT_F32, 4, spread=1.0)
    x, T, tokens = args(c)
    if dtype == wl.DT_BF16:
        x = x.bfloat16()
    g, h = cuda(c["g"], np.float32).double(), cuda(c["h"], np.float32).double()
    step = cuda(np.random.default_rng(5).choice([-1, 1], (B, V)), np.float32)
    eps = 2.0 ** -3 if dtype == wl.DT_BF16 else 2.0 ** -5
    up, down = (x.float() + eps * step).to(x.dtype), (x.float() - eps * step).to(x.dtype)

    def value(y):
        out = sfc.token_logprobs(y, T, tokens)
        return (g * out.logprobs.double()).sum() + (h * out.entropy.double()).sum()

    y = x.detach().requires_grad_()
    out = sfc.token_logprobs(y, T, tokens)
    (grad,) = torch.autograd.grad([out.logprobs, out.entropy], y, [g.float(), h.float()])
    slope = (grad.double() * (up.double() - down.double())).sum()
    # third derivatives along a unit direction: 8 / T^3 of a log-probability, 8 (1 + ln V) / T^3 of an entropy
    weight = float(g.abs().sum() + (h.abs() * 8).sum() * (1 + np.log(V))) * 8 / 0.5 ** 3
    d = float((up.double() - down.double()).abs().max()) / 2
    rounding = (2.0 ** -8 if dtype == wl.DT_BF16 else 2.0 ** -17) * float((grad.double() * (up.double() - down.double())).abs().sum())
    assert abs(float(value(up) - value(down) - slope)) <= weight * d ** 3 / 3 + rounding + 2.0 ** -14


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,V", [(5, 5003), (3, 100003), (320, 2003)])
@pytest.mark.parametrize("pad,offset,out_offset", [(1, 0, 0), (8, 8, 8), (3, 1, 1), (5, 0, 3), (16, 2, 0)])
def test_strides_and_alignments(dtype, B, V, pad, offset, out_offset):
    import top_support_capture_gb300 as sfc

    c = make(B, V, 3, dtype, pad + offset)
    ref, a = reference(c, 9), args(c, pad=pad, offset=offset)
    out = sfc.token_logprobs(*a, top=9, keep_stats=True)
    check_values(c, ref, out, 9)
    buf = torch.full((B * (V + pad) + out_offset,), 7.0, dtype=a[0].dtype, device="cuda")
    grad = buf[out_offset:].view(B, V + pad)[:, :V]
    sfc.token_logprobs_backward(*a, out.row_stats, cuda(c["g"], np.float32), cuda(c["h"], np.float32), grad=grad)
    check_grad(c, ref, oracle.token_logprobs_gradient(c["l"], dtype, c["T"], c["tokens"], c["g"], c["h"]), grad)
    assert (buf[:out_offset] == 7).all() and (buf[out_offset:].view(B, V + pad)[:, V:] == 7).all()


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("V", [2053, 40961])
@pytest.mark.parametrize("B", [14, 170])
def test_masked_and_extreme_logits(dtype, V, B):
    import top_support_capture_gb300 as sfc

    K = 12
    c = make(B, V, 3, dtype, 1)
    l = oracle.widen_logits(c["l"], dtype).astype(np.float32)
    c["tokens"][:] = [5, -1, 100]
    l[0, 300:] = -np.inf
    l[1, 300:] = LOW
    l[2, :] = LOW
    l[3, :] = -np.inf
    l[4, 2000] = np.nan
    l[5, 7] = np.inf
    l[6, 100] = -np.inf  # a given token
    l[7, 8:] = -np.inf   # fewer tokens than alternatives
    l[8, :] = -np.inf
    l[8, 1999] = LOW     # one token, of the lowest value
    c["tokens"][9, 2] = V
    c["tokens"][10, 0] = -2
    l[11, :] = 0.0       # all tied
    l[12, :] = -np.inf
    l[12, V - 1] = 60.0
    l[13, :] = np.where(np.arange(V) % 2 == 0, 0.0, -0.0)  # zeros of both signs tie
    c["l"] = as_input(l, dtype)
    ref = reference(c, K)
    assert list(ref.row_status[:14]) == [0, 0, 0, -1, -1, -1, 0, 0, 0, -1, -1, 0, 0, 0]
    a = args(c)
    out = sfc.token_logprobs(*a, top=K)
    check_values(c, ref, out, K)
    assert out.logprobs[6, 2] == -np.inf and out.top_ids[7, 8] == -1 and out.entropy[12] == 0
    want = oracle.token_logprobs_gradient(c["l"], dtype, c["T"], c["tokens"], c["g"], c["h"])
    x = a[0].detach().requires_grad_()
    two = sfc.token_logprobs(x, *a[1:], top=K)
    (grad,) = torch.autograd.grad([two.logprobs, two.entropy], x, [cuda(c["g"], np.float32), cuda(c["h"], np.float32)])
    check_grad(c, ref, want, grad)
    bad = torch.from_numpy(ref.row_status == -1).cuda()
    assert torch.isnan(out.logprobs[bad]).all() and torch.isnan(out.top_logprobs[bad]).all() and (out.top_ids[bad] == -1).all()
    assert not grad[bad].any()


def test_bad_temperatures():
    import top_support_capture_gb300 as sfc

    c = make(6, 100, 2, wl.DT_F32, 2)
    c["T"][:] = [0, -1, np.inf, np.nan, 1e-3, 1e4]
    ref = reference(c, 3)
    assert list(ref.row_status) == [-1, -1, -1, -1, 0, 0]
    check_values(c, ref, sfc.token_logprobs(*args(c), top=3), 3)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,V", [(2, 151936), (2, 50021), (350, 20000)])
@pytest.mark.parametrize("pattern", ["constant", "ascending", "descending", "few levels", "one thread", "lowest"])
def test_alternatives_of_patterned_rows(dtype, B, V, pattern):
    """Rows whose largest logits are tied, ordered, or all seen by the same thread: the pool overflows or nearly does."""
    import top_support_capture_gb300 as sfc

    K = 64
    rng = np.random.default_rng(0)
    i = np.arange(V)
    l = {"constant": np.full(V, 1.5), "ascending": i / V * 8, "descending": -i / V * 8, "few levels": rng.integers(0, 3, V),
         # vectors of 8 or 4 elements every 256 or 512 of them: the same thread of a CTA, whatever its size
         "one thread": np.where((i // (8 if dtype == wl.DT_BF16 else 4)) % 512 == 5, 4 + rng.random(V), rng.random(V)),
         "lowest": np.where(rng.random(V) < 1e-4, rng.random(V), LOW)}[pattern]
    l = np.broadcast_to(l.astype(np.float32), (B, V)).copy()
    l[1::2] += 0 if pattern == "lowest" else 0.25
    c = dict(l=as_input(l, dtype), dtype=dtype, T=np.full(B, 0.8, np.float32), tokens=np.zeros((B, 1), np.int32))
    some = {**c, **{k: c[k][:2] for k in ("l", "T", "tokens")}}
    ref, out = reference(some, K), sfc.token_logprobs(*args(c), top=K)
    first = type(out)(*(t if t is None else t[:2] for t in out))
    check_values(some, ref, first, K)
    assert torch.equal(out.top_ids, out.top_ids[:2].repeat(B // 2, 1))  # every row like the first two


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_steep_and_flat_rows(dtype):
    """Rows of one certain token, and of nearly equal ones, at temperatures that make them steeper or flatter."""
    import top_support_capture_gb300 as sfc

    c = make(4, 30000, 2, dtype, 6)
    l = oracle.widen_logits(c["l"], dtype).astype(np.float32)
    l[0, 17] = 300.0
    l[1] *= 20
    l[2] *= 1e-3
    c["T"][:] = [1.0, 0.05, 100.0, 3e-3]
    c["l"] = as_input(l, dtype)
    ref, a = reference(c, 5), args(c)
    check_values(c, ref, sfc.token_logprobs(*a, top=5), 5)
    x = a[0].detach().requires_grad_()
    out = sfc.token_logprobs(x, *a[1:])
    (grad,) = torch.autograd.grad([out.logprobs, out.entropy], x, [cuda(c["g"], np.float32), cuda(c["h"], np.float32)])
    check_grad(c, ref, oracle.token_logprobs_gradient(c["l"], dtype, c["T"], c["tokens"], c["g"], c["h"]), grad)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_a_very_long_row(dtype):
    import top_support_capture_gb300 as sfc

    c = make(2, 3_000_017, 2, dtype, 12)
    ref, a = reference(c, 64), args(c, pad=3, offset=1)
    out = sfc.token_logprobs(*a, top=64, keep_stats=True)
    check_values(c, ref, out, 64)
    grad = sfc.token_logprobs_backward(*a, out.row_stats, cuda(c["g"], np.float32), cuda(c["h"], np.float32))
    check_grad(c, ref, oracle.token_logprobs_gradient(c["l"], dtype, c["T"], c["tokens"], c["g"], c["h"]), grad)


@pytest.mark.parametrize("shift", [-3e4, 1e6])
def test_shifted_logits(shift):
    """A constant added to a row changes nothing: the exponents' reference is far from 0 there."""
    import top_support_capture_gb300 as sfc

    c = make(5, 20011, 3, wl.DT_F32, 13)
    c["l"] = (c["l"] + np.float32(shift)).astype(np.float32)
    ref, a = reference(c, 7), args(c)
    x = a[0].detach().requires_grad_()
    out = sfc.token_logprobs(x, *a[1:], top=7)
    check_values(c, ref, out, 7)
    (grad,) = torch.autograd.grad([out.logprobs, out.entropy], x, [cuda(c["g"], np.float32), cuda(c["h"], np.float32)])
    check_grad(c, ref, oracle.token_logprobs_gradient(c["l"], c["dtype"], c["T"], c["tokens"], c["g"], c["h"]), grad)


def test_differentiable_on_another_stream():
    import top_support_capture_gb300 as sfc

    c = make(4, 200_003, 3, wl.DT_BF16, 16)
    ref, a = reference(c, 4), args(c)
    g, h = cuda(c["g"], np.float32), cuda(c["h"], np.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x = a[0].detach().requires_grad_()
    out = sfc.token_logprobs(x, *a[1:], top=4, stream=side)
    with torch.cuda.stream(side):
        (grad,) = torch.autograd.grad([out.logprobs, out.entropy], x, [g, h])
    torch.cuda.current_stream().wait_stream(side)
    check_values(c, ref, out, 4)
    check_grad(c, ref, oracle.token_logprobs_gradient(c["l"], c["dtype"], c["T"], c["tokens"], c["g"], c["h"]), grad)


def test_saved_tensors_that_are_moved():
    """Hooks that keep what a backward needs elsewhere bring rows back that lie next to each other."""
    import top_support_capture_gb300 as sfc

    c = make(5, 5003, 3, wl.DT_BF16, 15)
    ref, a = reference(c), args(c, pad=13, offset=2)
    x = a[0].detach().requires_grad_()
    with torch.autograd.graph.save_on_cpu():
        out = sfc.token_logprobs(x, *a[1:], top=2)
    (grad,) = torch.autograd.grad([out.logprobs, out.entropy], x, [cuda(c["g"], np.float32), cuda(c["h"], np.float32)])
    check_grad(c, ref, oracle.token_logprobs_gradient(c["l"], c["dtype"], c["T"], c["tokens"], c["g"], c["h"]), grad)


def test_streams_graphs_and_repeats():
    import top_support_capture_gb300 as sfc

    c = make(6, 40960, 2, wl.DT_BF16, 9)
    a, g = args(c), cuda(c["g"], np.float32)
    same = lambda p, q: all(torch.equal(x, y) for x, y in zip(p, q) if x is not None)
    first = sfc.token_logprobs(*a, top=7, keep_stats=True)
    assert same(first, sfc.token_logprobs(*a, top=7, keep_stats=True))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sfc.token_logprobs(*a, top=7, keep_stats=True, stream=side)
    grad = sfc.token_logprobs_backward(*a, other.row_stats, g, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert same(first, other) and torch.equal(grad, sfc.token_logprobs_backward(*a, first.row_stats, g))
    graphs = []
    for top in (7, 3):  # two graphs over the same inputs
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = sfc.token_logprobs(*a, top=top, keep_stats=True)
            grad = sfc.token_logprobs_backward(*a, held.row_stats, g)
        graphs.append((graph, held, grad, top))
    a[0].mul_(0.5)  # new inputs in the same place
    c["l"] = a[0].view(torch.int16).cpu().numpy().view(np.uint16)
    streams = [torch.cuda.Stream() for _ in graphs]
    for s, (graph, *_) in zip(streams, graphs):  # side by side
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                graph.replay()
    torch.cuda.synchronize()
    for _, held, grad, top in graphs:
        ref = reference(c, top)
        check_values(c, ref, held, top)
        check_grad(c, ref, oracle.token_logprobs_gradient(c["l"], wl.DT_BF16, c["T"], c["tokens"], c["g"]), grad)


def test_rows_past_32_bit_offsets():
    import top_support_capture_gb300 as sfc

    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    V, B, last = 262144, 8200, 2
    c = make(last, V, 2, wl.DT_BF16, 5)
    big = torch.zeros((B, V), dtype=torch.bfloat16, device="cuda")
    big[-last:] = dev_logits(c["l"], wl.DT_BF16)
    T, tokens = torch.ones(B, device="cuda"), torch.zeros((B, 2), dtype=torch.int32, device="cuda")
    T[-last:], tokens[-last:] = cuda(c["T"], np.float32), cuda(c["tokens"], np.int32)
    g = torch.zeros((B, 2), device="cuda")
    g[-last:] = cuda(c["g"], np.float32)
    out = sfc.token_logprobs(big, T, tokens, top=4, keep_stats=True)
    ref = reference(c, 4)
    check_values(c, ref, type(out)(*(t[-last:] for t in out)), 4)
    assert not out.row_status.any() and (out.top_ids[:-last] == torch.arange(4, device="cuda")).all()
    grad = sfc.token_logprobs_backward(big, T, tokens, out.row_stats, g)
    check_grad(c, ref, oracle.token_logprobs_gradient(c["l"], wl.DT_BF16, c["T"], c["tokens"], c["g"]), grad[-last:])
    assert not grad[:-last].any()


# Rows in one CTA of 128 or 256 threads, up to the longest of each and above it.
@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("B,vectors", [(320, 60), (320, 1369), (320, 4000), (310, 7000), (310, 7001), (306, 18992), (306, 54721)])
def test_many_rows(dtype, B, vectors):
    import top_support_capture_gb300 as sfc

    V, K = vectors * (8 if dtype == wl.DT_BF16 else 4) + 3, 30
    gen = torch.Generator("cuda").manual_seed(vectors)
    x = torch.randn((B, V), generator=gen, device="cuda").mul_(3).to(torch.bfloat16 if dtype == wl.DT_BF16 else torch.float32)
    x[1, 1000:] = -float("inf")
    x[2, ::2] = -float("inf")
    x[3] = x[3].round()  # ties
    rng = np.random.default_rng(vectors)
    T, tokens = rng.uniform(0.5, 1.7, B).astype(np.float32), rng.integers(-1, V, (B, 2)).astype(np.int32)
    out = sfc.token_logprobs(x, cuda(T, np.float32), cuda(tokens, np.int32), top=K)
    assert not out.row_status.any() and torch.isfinite(out.entropy).all()
    rows = np.unique(np.r_[0, 1, 2, 3, B - 1, rng.integers(0, B, 4)])
    at = torch.from_numpy(rows).cuda()
    l = x[at].view(torch.int16).cpu().numpy().view(np.uint16) if dtype == wl.DT_BF16 else x[at].cpu().numpy()
    some = dict(l=l, dtype=dtype, T=T[rows], tokens=tokens[rows])
    check_values(some, reference(some, K), type(out)(*(t if t is None else t[at] for t in out)), K)
    again = sfc.token_logprobs(x, cuda(T, np.float32), cuda(tokens, np.int32), top=K)
    assert all(torch.equal(p, q) for p, q in zip(out[:5], again[:5]))  # whatever the order in which the slices' arrive
