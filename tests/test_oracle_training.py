"""Pins of the distillation, replay-gradient and verification oracles (CPU)."""
import numpy as np
import pytest

import oracle
from oracle.verify import waits
from top_support_capture_gb300 import workloads as wl


def _teacher(rng, B, V, W):
    ids = np.stack([rng.choice(V, W, replace=False) for _ in range(B)]).astype(np.int32)
    y = rng.standard_normal((B, W)).astype(np.float32)
    return ids, y - np.log(np.exp(y).sum(1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("normalise", [False, True])
def test_distill_gradient_against_differences(normalise):
    rng = np.random.default_rng(3)
    B, V, W = 3, 11, 4
    l, T = rng.standard_normal((B, V)).astype(np.float32), np.array([0.7, 1.0, 1.6], np.float32)
    ids, y = _teacher(rng, B, V, W)
    lens, g = np.array([4, 2, 1], np.int32), np.array([1.0, -0.5, 2.0])
    run = lambda x: oracle.distill(x, wl.DT_F32, T, ids, y, lens, W, g, normalise)
    grad, h = run(l).grad, 2.0 ** -7
    for r in range(B):
        for j in range(V):
            d = np.zeros_like(l)
            d[r, j] = h
            up, down = (l + d).astype(np.float32), (l - d).astype(np.float32)
            slope = (run(up).loss[r] - run(down).loss[r]) / (float(up[r, j]) - float(down[r, j]))
            # central difference: h^2 / 6 times a third derivative of at most (2 / T)^3
            assert abs(slope * g[r] - grad[r, j]) <= abs(g[r]) * h * h / 6 * (2 / T[r]) ** 3 + 1e-7


def test_distill_closed_forms():
    l = np.zeros((1, 8), np.float32)
    ids, one = np.array([[3, 5]], np.int32), np.ones(1)
    # a uniform student against a teacher of two halves: ln 8 - ln 2; the gradient p - t
    res = oracle.distill(l, wl.DT_F32, [1.0], ids, np.log(np.full((1, 2), 0.5, np.float32)), [2], 2, one)
    assert abs(res.loss[0] - np.log(4)) < 1e-7
    want = np.full(8, 1 / 8)
    want[[3, 5]] -= 0.5
    np.testing.assert_allclose(res.grad[0], want, atol=1e-7)
    # a student equal to a teacher over the whole vocabulary: no loss, no gradient
    rng = np.random.default_rng(0)
    l = rng.standard_normal((1, 8)).astype(np.float32)
    res = oracle.distill(l, wl.DT_F32, [1.5], np.arange(8, dtype=np.int32)[None], l, [8], 8, one, normalise=True)
    assert abs(res.loss[0]) < 1e-12 and np.abs(res.grad).max() < 1e-12


def test_replay_gradient_against_differences():
    rng = np.random.default_rng(4)
    B, V, W = 3, 9, 5
    l, T = rng.standard_normal((B, V)).astype(np.float32), np.array([0.8, 1.0, 1.3], np.float32)
    ids, _ = _teacher(rng, B, V, W)
    lens, tok = np.array([5, 3, 1], np.int32), np.array([ids[0, 2], ids[1, 0], ids[2, 0]], np.int32)
    g, G = rng.standard_normal(B), rng.standard_normal((B, W))

    def value(x, r):
        res = oracle.replay_logprob(x, wl.DT_F32, T, ids, lens, W, tok)
        return g[r] * res.token_logprob[r] + (G[r, :lens[r]] * res.support_logprobs[r, :lens[r]]).sum()

    grad, _ = oracle.replay_gradient(l, wl.DT_F32, T, ids, lens, W, tok, g, G)
    h = 2.0 ** -7
    for r in range(B):
        for j in range(V):
            d = np.zeros_like(l)
            d[r, j] = h
            up, down = (l + d).astype(np.float32), (l - d).astype(np.float32)
            slope = (value(up, r) - value(down, r)) / (float(up[r, j]) - float(down[r, j]))
            scale = abs(g[r]) + np.abs(G[r]).sum()
            assert abs(slope - grad[r, j]) <= scale * h * h / 6 * (2 / T[r]) ** 3 + 1e-7


def test_waits_are_the_words_of_philox():
    """Token 4 k + w reads word w of the block at counter (2^31 + k, row, step)."""
    e = waits(np.arange(12), 7, 0x1122334455667788, 0x99AABBCCDDEEFF00)
    for i in range(12):
        block = oracle.philox4x32_10(np.uint32(2 ** 31 + i // 4), 7, 0xDDEEFF00, 0x99AABBCC, 0x55667788, 0x11223344)
        assert e[i] == -np.log((2.0 * float(int(block[i % 4]) >> 9) + 1) * 2.0 ** -24)


def _rounds(B, V, D, seed):
    """One target and draft distribution for B requests, drafts drawn from the draft's rows."""
    rng = np.random.default_rng(seed)
    t, d = rng.standard_normal((D + 1, V)).astype(np.float32), rng.standard_normal((D, V)).astype(np.float32)
    q = np.exp(d.astype(np.float64))
    q /= q.sum(1, keepdims=True)
    drafts = np.stack([rng.choice(V, size=B, p=q[j]) for j in range(D)], 1).astype(np.int32)
    return t, d, drafts, rng.random((B, D)).astype(np.float32)


def test_emitted_tokens_follow_the_target():
    """The first token of every request is distributed as the target's first row (chi-square)."""
    B, V, D = 4000, 5, 2
    t, d, drafts, u = _rounds(B, V, D, 11)
    res = oracle.verify_drafts(np.broadcast_to(t, (B, D + 1, V)), np.broadcast_to(d, (B, D, V)), wl.DT_F32, drafts, u,
                               np.ones(B), 5, 9)
    p = np.exp(t[0].astype(np.float64))
    p /= p.sum()
    seen = np.bincount(res.tokens[:, 0], minlength=V)
    assert ((seen - B * p) ** 2 / (B * p)).sum() < 23.5  # 4 degrees of freedom, 1e-4
    # the second token of the requests that accepted the first draft follows the second row
    ok = res.accepted >= 1
    p = np.exp(t[1].astype(np.float64))
    p /= p.sum()
    seen = np.bincount(res.tokens[ok, 1], minlength=V)
    assert ((seen - ok.sum() * p) ** 2 / (ok.sum() * p)).sum() < 23.5


def test_supports_and_rows_agree():
    """Supports that hold the whole vocabulary give what the full rows give."""
    B, V, D = 40, 6, 3
    t, d, drafts, u = _rounds(B, V, D, 2)
    full = oracle.verify_drafts(np.broadcast_to(t, (B, D + 1, V)), np.broadcast_to(d, (B, D, V)), wl.DT_F32, drafts, u,
                                np.ones(B), 5, 9)
    lsm = lambda x: x - np.log(np.exp(x).sum(-1, keepdims=True))
    rows = lambda x, k: np.broadcast_to(x, (B, k, V))
    ids = np.arange(V, dtype=np.int32)
    res = oracle.verify_supports(rows(ids, D + 1), rows(lsm(t.astype(np.float64)), D + 1), np.full((B, D + 1), V),
                                 rows(ids, D), rows(lsm(d.astype(np.float64)), D), np.full((B, D), V), drafts, u, 5, 9)
    np.testing.assert_array_equal(res.tokens, full.tokens)
    np.testing.assert_array_equal(res.accepted, full.accepted)


def test_certain_and_greedy_drafts():
    l = np.array([[[0.0, 3.0, 1.0]] * 3], np.float32)
    one, u = np.ones(1), np.array([[0.5, 0.99]], np.float32)
    # certain drafts of probability 0.84: 0.5 < 0.84 accepts, 0.99 refuses, and the next token is another
    res = oracle.verify_drafts(l, None, wl.DT_F32, np.array([[1, 1]]), u, one, 1, 2)
    assert res.accepted[0] == 1 and res.tokens[0, 0] == 1 and res.tokens[0, 1] in (0, 2) and res.tokens[0, 2] == -1
    # greedy rows accept the largest and emit it
    res = oracle.verify_drafts(l, None, wl.DT_F32, np.array([[1, 0]]), u, 0 * one, 1, 2, greedy_t0=True)
    assert res.accepted[0] == 1 and list(res.tokens[0]) == [1, 1, -1] and list(res.token_logprobs[0]) == [0, 0, 0]
    assert oracle.verify_drafts(l, None, wl.DT_F32, np.array([[1, 0]]), u, 0 * one, 1, 2).row_status[0] == oracle.ROW_BADPARAM
