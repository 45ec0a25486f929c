"""Pins of the oracles of whole-vocabulary log-probabilities, the policy loss and gradient clipping (CPU)."""
import math

import numpy as np
import pytest

import oracle
from top_support_capture_gb300 import workloads as wl


def differences(value, l, r, h=2.0 ** -7):
    """Central differences of value(l)[r] along the row's logits."""
    out = np.zeros(l.shape[1])
    for j in range(l.shape[1]):
        d = np.zeros_like(l)
        d[r, j] = h
        up, down = (l + d).astype(np.float32), (l - d).astype(np.float32)
        out[j] = (value(up) - value(down)) / (float(up[r, j]) - float(down[r, j]))
    return out


def test_gradient_against_differences():
    rng = np.random.default_rng(3)
    B, V, M = 3, 9, 3
    l, T = rng.standard_normal((B, V)).astype(np.float32), np.array([0.7, 1.0, 1.6], np.float32)
    tokens = np.array([[0, 4, -1], [8, 8, 2], [5, -1, -1]], np.int32)  # one of them twice
    g, h = rng.standard_normal((B, M)), rng.standard_normal(B)
    grad = oracle.token_logprobs_gradient(l, wl.DT_F32, T, tokens, g, h).grad
    for r in range(B):
        def value(x):
            out = oracle.token_logprobs(x, wl.DT_F32, T, tokens)
            return (g[r] * out.logprobs[r]).sum() + h[r] * out.entropy[r]

        # h^2 / 6 times a third derivative: of a log-probability at most (2 / T)^3, of the entropy 8 (1 + ln V) times that
        third = (np.abs(g[r]).sum() + abs(h[r]) * 8 * (1 + math.log(V))) * (2 / T[r]) ** 3
        assert np.abs(differences(value, l, r) - grad[r]).max() <= 2.0 ** -14 / 6 * third + 1e-7


def test_closed_forms():
    l = np.zeros((2, 8), np.float32)
    l[1, 3:] = -np.inf
    out = oracle.token_logprobs(l, wl.DT_F32, [1.0, 0.5], np.array([[2, -1], [1, 5]]), top=4)
    np.testing.assert_allclose(out.entropy, [math.log(8), math.log(3)], atol=1e-12)
    np.testing.assert_allclose(out.logprobs, [[-math.log(8), 0], [-math.log(3), -np.inf]], atol=1e-12)
    assert out.top_ids.tolist() == [[0, 1, 2, 3], [0, 1, 2, -1]]  # ties by id; masked tokens are no alternatives
    assert out.top_logprobs[1, 3] == -np.inf and not out.row_status.any()
    # the entropy of a uniform row is at its maximum
    assert np.abs(oracle.token_logprobs_gradient(l, wl.DT_F32, [1.0, 0.5], np.array([[-1], [-1]]), [[0], [0]], [1, 1]).grad).max() < 1e-12
    bad = oracle.token_logprobs(l, wl.DT_F32, [1.0, 0.0], np.array([[8], [0]]))
    assert bad.row_status.tolist() == [-1, -1] and np.isnan(bad.entropy).all()


@pytest.mark.parametrize("weight", [0.0, 0.3])
def test_policy_gradient_against_differences(weight):
    rng = np.random.default_rng(5)
    B, V = 6, 7
    l, T = rng.standard_normal((B, V)).astype(np.float32), rng.uniform(0.6, 1.5, B).astype(np.float32)
    tokens = rng.integers(0, V, B)
    lp = oracle.token_logprobs(l, wl.DT_F32, T, tokens).logprobs[:, 0]
    # ratios inside, above and below the range, for advantages of both signs
    old, A = lp - np.log([1.0, 1.6, 0.5, 1.0, 1.6, 0.5]), np.array([1.0, 1.5, 2.0, -1.0, -1.5, -2.0])
    g = rng.standard_normal(B)
    for o in (None, old):
        run = lambda x: oracle.policy_loss(x, wl.DT_F32, T, tokens, A, g, o, 0.2, 0.28, weight)
        out = run(l)
        if o is not None:
            assert (out.slope == 0).tolist() == [False, True, False, False, False, True]
        for r in range(B):
            third = abs(g[r]) * (abs(A[r]) * 2 + weight * 8 * (1 + math.log(V))) * (4 / T[r]) ** 3
            assert np.abs(differences(lambda x: run(x).loss[r] * g[r], l, r) - out.grad[r]).max() <= 2.0 ** -14 / 6 * third + 1e-7


def test_policy_rows():
    l = np.zeros((6, 4), np.float32)
    l[3, 1] = np.nan
    l[4, 2] = -np.inf
    out = oracle.policy_loss(l, wl.DT_F32, np.ones(6), [0, -1, 4, -1, 2, 2], np.array([1, 1, 1, 1, 1, np.inf]), np.ones(6))
    assert out.row_status.tolist() == [0, 0, -1, 0, 0, -1]
    assert out.loss[0] == math.log(4) and out.loss[1] == 0 and np.isnan(out.loss[2]) and out.loss[4] == np.inf
    np.testing.assert_allclose(out.grad[0], [-0.75, 0.25, 0.25, 0.25], atol=1e-12)
    assert not out.grad[1:].any()


def test_clip():
    a, b = np.array([3.0, 0.0]), np.array([[4.0]])
    assert oracle.grad_norm([a, b]) == 5.0
    assert oracle.clip_scale(5.0, 10.0) == 1.0 and oracle.clip_scale(5.0, math.inf) == 1.0 and oracle.clip_scale(0.0, 0.0) == 0.0
    assert oracle.clip_scale(5.0, 1.0) == 1.0 / (5.0 + 1e-6) and oracle.clip_scale(math.inf, 1.0) == 0.0
