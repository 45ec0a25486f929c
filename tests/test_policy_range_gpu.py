"""The policy step over the whole range of its exponents |x| / T: rows whose masked logits hold a finite fill, low temperatures,
large logits. Tolerances as in test_policy_gpu, and one that matters where T is small: an exponential below the smallest normal
number 2^-126 is flushed to 0, so that an entry p (G + h (ln p + H)) / T of such a token is off by 2^-126 (|G| + |h| (|ln p| + H)) / T,
with |ln p| < 127 ln 2 + ln V < 110 there. Log-probabilities and entropies are also those of token_logprobs.

By 16-byte vectors a row: kept slices of 128, 256, 512 and 1024 threads, and rows that are read again."""
import numpy as np
import pytest

import oracle
from top_support_capture_gb300 import workloads as wl
from test_distill_gpu import HALF, _cuda, as_input  # noqa: F401 (the fixture)
from test_policy_gpu import call, reference
from test_token_logprobs_gpu import args, check_values, close, grad_limit

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
VECTORS = [500, 10000, 20000, 45000, 100000, 110000]
LOW = np.float32(-3.3895313892515355e38)  # bfloat16's lowest value


def make(l, dtype, T, tokens, clipped, weight, seed=0):
    """A case of the logits l at T; clipped: ratios from 0.6 to 1.6, away from the borders."""
    rng = np.random.default_rng(seed)
    B = len(l)
    c = dict(l=as_input(l, dtype), dtype=dtype, T=np.broadcast_to(np.asarray(T, np.float32), (B,)).copy(),
             tokens=np.asarray(tokens, np.int32), A=rng.choice([-1, 1], B).astype(np.float32) * rng.uniform(0.5, 2, B).astype(np.float32),
             g=rng.uniform(0.5, 2, B).astype(np.float32), weight=weight, old=None)
    if clipped:
        lp = oracle.token_logprobs(c["l"], dtype, c["T"], c["tokens"]).logprobs[:, 0]
        c["old"] = (lp - rng.choice([0.0, 0.1, -0.1, 0.5, -0.5], B)).astype(np.float32)
    return c


def check(c, out):
    ref = reference(c)
    stats = oracle.token_logprobs(c["l"], c["dtype"], c["T"], c["tokens"])
    np.testing.assert_array_equal(out.row_status.cpu().numpy(), ref.row_status)
    H, lp = ref.entropy, np.abs(ref.logprobs)
    off_lp = 104 + 4 * H + 6 * stats.ln_mass + 5 * lp  # half steps
    off_H = 104 + 106 * H + stats.ln_mass + 4 * stats.spread
    close(out.logprobs, ref.logprobs, HALF * off_lp)
    close(out.entropy, ref.entropy, HALF * off_H)
    off_rho = 0.0 * lp if c["old"] is None else off_lp + 2 * np.abs(c["old"]) + 8
    size = np.abs(ref.slope) * (off_lp if c["old"] is None else off_rho)
    close(out.loss, ref.loss, HALF * (size + abs(c["weight"]) * (off_H + 2 * H) + 4 * np.abs(ref.loss)))
    got = out.grad_logits.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    flushed = 2.0 ** -126 * (np.abs(ref.slope) + abs(c["weight"]) * (110 + H)) * np.abs(c["g"]) / c["T"].astype(np.float64)
    over = np.abs(got - ref.grad) - grad_limit(c, stats.far, ref.grad, ref.grad_scale, off_rho[:, None]) - flushed[:, None]
    assert over.max() <= 0, (np.unravel_index(over.argmax(), over.shape), over.max())
    return ref


def check_all(c, layout={}):
    """The step against the oracle, beside the scores of the same rows; returns the oracle's."""
    import top_support_capture_gb300 as sfc

    ref = check(c, call(c, layout=layout))
    assert not ref.row_status.any()
    score = dict(c, tokens=c["tokens"][:, None])
    check_values(score, oracle.token_logprobs(c["l"], c["dtype"], c["T"], score["tokens"]), sfc.token_logprobs(*args(score, **layout)))
    return ref


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("vectors", VECTORS)
@pytest.mark.parametrize("clipped", [True, False])
def test_rows_masked_by_a_finite_fill(dtype, vectors, clipped):
    """Four tokens are left: nearly every thread sees nothing but the fill."""
    V = vectors * (8 if dtype == wl.DT_BF16 else 4) + 3
    rng = np.random.default_rng(vectors)
    fills, temperatures = [-1e4, -1e9, -1e10, -1e12, -1e15, LOW, -np.inf], [1.0, 0.3, 0.1]
    if vectors > 20000:  # (the rows are long)
        temperatures = [0.3]
    cases = [(f, t) for f in fills for t in temperatures]
    l = np.empty((len(cases), V), np.float32)
    tokens = []
    for r, (fill, _) in enumerate(cases):
        l[r] = fill
        allowed = rng.choice(V, 4, replace=False)
        l[r, allowed] = rng.standard_normal(4)
        tokens.append(allowed[0])
    check_all(make(l, dtype, [t for _, t in cases], tokens, clipped, 0.02))


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("vectors", [500, 10000, 20000, 110000])
@pytest.mark.parametrize("clipped", [True, False])
def test_low_temperatures(dtype, vectors, clipped):
    V = vectors * (8 if dtype == wl.DT_BF16 else 4) + 3
    T = [1e-2, 1e-4, 1e-6, 1e-7, 3e-8, 1e-8, 1e-9, 1e-10, 1e-12, 1e-16, 1e-18, 1e-20, 1e-25]
    l = (np.random.default_rng(vectors).standard_normal((len(T), V)) * 3).astype(np.float32)
    tokens = l.argmax(1)
    l[np.arange(len(T)), tokens - 1] = l.max(1)  # tied with another
    check_all(make(l, dtype, T, tokens, clipped, 0.02))


@pytest.mark.parametrize("scale", [1e5, 1e7, 1e9, 1e10, 1e13, 1e17, 1e25, 1e37])
def test_large_logits(scale):
    for clipped in (True, False):
        l = (np.random.default_rng(3).standard_normal((4, 20011)) * scale).astype(np.float32)
        l[1] += np.float32(scale)
        check_all(make(l, wl.DT_F32, 1.0, l.argmax(1), clipped, 0.02))


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("fill", [-1e9, -1e12, LOW])
def test_the_largest_logit_beside_the_vectors(dtype, fill):
    """The row's largest logits lie in its unaligned head and its tail, and everything else is masked: the threads' references
    and the row's are far apart."""
    V = 5003
    l = np.full((4, V), fill, np.float32)
    l[:, :2] = [[1.0, 0.5], [2.0, -1.0], [-3.0, -3.0], [0.0, 4.0]]
    l[2:, V - 1] = [1.0, 3.5]
    check_all(make(l, dtype, [1.0, 0.1, 0.3, 1e-9], [0, 1, V - 1, 1], False, 0.02), layout=dict(pad=5, offset=1))
