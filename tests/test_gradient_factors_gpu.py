"""Gradients over the whole vocabulary whose factors are near the largest number, or past it. Tolerances as in
test_policy_range_gpu."""
import numpy as np
import pytest

import oracle
from top_support_capture_gb300 import workloads as wl
from test_distill_gpu import _cuda, as_input, cuda  # noqa: F401 (the fixture)
from test_policy_gpu import call
from test_policy_range_gpu import check
from test_token_logprobs_gpu import args, grad_limit

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
LOW = np.float32(-3.3895313892515355e38)  # bfloat16's lowest value


def steep(dtype, T, seed):
    """Rows of a few likely tokens, the others improbable or masked, whose logits are of the temperature's size."""
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((6, 2053)).astype(np.float32) * 20
    l[3] = 0.0
    l[4, 100:] -= 500
    l = (l.astype(np.float64) * T).astype(np.float32)
    l[1, 200:] = -np.inf
    l[2, 300:] = LOW
    l[5, :] = -np.inf
    l[5, [3, 700]] = 0.0
    return as_input(l, dtype), np.where(np.arange(6) == 5, 3, l.argmax(1)).astype(np.int32)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("T", [1e-30, 1e-37, 1.5e-38, 6e-39])
def test_factors_near_the_largest_number(dtype, T):
    """1 / T takes an entry's factors close to the end of the range, where their products with improbable tokens' exponents pass
    it; the gradients themselves are within it."""
    import top_support_capture_gb300 as sfc

    l, tokens = steep(dtype, np.float32(T), 5)
    B = len(tokens)
    c = dict(l=l, dtype=dtype, T=np.full(B, T, np.float32), tokens=tokens, A=np.full(B, 0.25, np.float32), g=np.full(B, 0.9, np.float32),
             weight=0.8, old=None)
    ref = check(c, call(c))
    assert np.abs(ref.grad).max() < 3e38 and not ref.row_status.any()
    score = dict(c, tokens=tokens[:, None])
    a = args(score)
    out = sfc.token_logprobs(*a, keep_stats=True)
    want = oracle.token_logprobs_gradient(l, dtype, c["T"], score["tokens"], np.full((B, 1), 0.3), np.full(B, -0.7))
    grad = sfc.token_logprobs_backward(*a, out.row_stats, cuda(np.full((B, 1), 0.3), np.float32), cuda(np.full(B, -0.7), np.float32))
    stats = oracle.token_logprobs(l, dtype, c["T"], score["tokens"])
    flushed = 2.0 ** -126 * (0.3 + 0.7 * (110 + stats.entropy)) / c["T"].astype(np.float64)  # (see test_policy_range_gpu)
    got = grad.float().cpu().numpy().astype(np.float64)
    over = np.abs(got - want.grad) - grad_limit(c, stats.far, want.grad, want.grad_scale) - flushed[:, None]
    assert np.isfinite(got).all() and over.max() <= 0, (np.unravel_index(over.argmax(), over.shape), over.max())


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_factors_past_the_largest_number(dtype):
    """At temperatures whose inverse is not a float32 the factors are held: certain tokens' rows have the gradient 0 that they
    have at every temperature, and nothing becomes NaN."""
    import top_support_capture_gb300 as sfc

    B, V = 3, 2053
    l = np.random.default_rng(1).standard_normal((B, V)).astype(np.float32)
    l[1, 1000:] = -np.inf
    l[2, 1:] = -np.inf
    tokens = l.argmax(1).astype(np.int32)
    l[np.arange(B), tokens] += 4
    l = as_input(l, dtype)
    T, g = np.full(B, 1e-39, np.float32), np.full(B, 3.0, np.float32)
    for A in (1.0, -1.0):
        out = call(dict(l=l, dtype=dtype, T=T, tokens=tokens, A=np.full(B, A, np.float32), g=g, weight=0.5, old=None))
        assert not out.row_status.any() and not torch.isnan(out.grad_logits).any() and not out.grad_logits.isinf().any()
    a = args(dict(l=l, dtype=dtype, T=T, tokens=tokens[:, None]))
    grad = sfc.token_logprobs_backward(*a, sfc.token_logprobs(*a, keep_stats=True).row_stats, cuda(g[:, None], np.float32), cuda(g, np.float32))
    assert not torch.isnan(grad).any() and not grad.isinf().any()
