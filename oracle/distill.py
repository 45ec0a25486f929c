"""Float64 CPU oracle of the distillation loss and gradient, and of the replay's gradient.

TEST INFRASTRUCTURE, like the rest of this package. Formulas (z = l / T):
  distillation  t = exp(y), or softmax(y / T) over the row's entries; p = softmax(z) over the vocabulary;
                loss = sum t (ln t - ln p), gradient g (sum(t) p - t) / T
  replay        lp = log-softmax of z over the support S; with upstream gradients u of the members' lp the
                gradient is (u - exp(lp) sum u) / T on S, 0 elsewhere
Both come row by row from their definitions: the gradients from the Jacobian of the log-softmax, not from the
library's arrangement of the sums.
"""
from __future__ import annotations

import dataclasses

import numpy as np

from .replay import ROW_OUTSIDE, replay_row
from .sfc_oracle import ROW_BADPARAM, ROW_OK, ROW_OVERFLOW, widen_logits


@dataclasses.dataclass
class DistillResult:
    loss: np.ndarray  # float64 [B]; NaN on BADPARAM rows
    grad: np.ndarray  # float64 [B, V]
    row_status: np.ndarray  # int32 [B]
    grad_scale: np.ndarray  # float64 [B, V]: the sum of the magnitudes that a gradient entry is a difference of
    loss_scale: np.ndarray  # float64 [B]: the same for the loss


def _log_softmax(z):
    z = z - z.max()  # first: a row of the lowest values would lose the logarithm of its mass to rounding
    return z - np.log(np.exp(z).sum())


def distill_row(l, T, ids, y, n, W, g, normalise):
    """(status, loss, gradient, magnitudes of the loss, magnitudes of the gradient) of one row."""
    V = l.shape[0]
    zero = np.zeros(V)
    bad = (ROW_BADPARAM, np.nan, zero, 0.0, zero)
    if not (np.isfinite(T) and T > 0.0) or n < 0:
        return bad
    status = ROW_OVERFLOW if n > W else ROW_OK
    n = min(n, W)
    if n == 0:
        return status, 0.0, zero, 0.0, zero
    ids, y = np.asarray(ids[:n], np.int64), np.asarray(y[:n], np.float64)
    if ids.min() < 0 or ids.max() >= V or np.isnan(l).any() or np.isposinf(l).any() or not np.isfinite(l).any():
        return bad
    if np.isnan(y).any() or np.isposinf(y).any() or (normalise and not np.isfinite(y).any()):
        return bad
    ln_p = _log_softmax(l / T)
    ln_t = _log_softmax(y / T) if normalise else y
    t = np.exp(ln_t)
    on = t > 0
    with np.errstate(invalid="ignore"):
        loss = float(np.sum(t[on] * (ln_t[on] - ln_p[ids[on]])))
    # d ln p_i / d x_j = (delta_ij - p_j) / T
    p = np.exp(ln_p)
    grad = np.zeros(V)
    grad[ids] = -t
    mag = p * t.sum()
    grad += mag
    mag[ids] += t
    zrel = np.abs(l / T - (l / T).max())
    return status, loss, grad * g / T, float(np.sum(t[on] * (np.abs(ln_t[on]) + zrel[ids[on]])) + t.sum() * abs(ln_p.max())), mag * abs(g) / T


def distill(logits, dtype, temperature, teacher_ids, teacher_values, lengths, packed_width, grad_loss,
            normalise=False) -> DistillResult:
    L = widen_logits(logits, dtype)
    B, V = L.shape
    out = DistillResult(np.zeros(B), np.zeros((B, V)), np.zeros(B, np.int32), np.zeros((B, V)), np.zeros(B))
    T = np.asarray(temperature, np.float32).astype(np.float64)
    for r in range(B):
        out.row_status[r], out.loss[r], out.grad[r], out.loss_scale[r], out.grad_scale[r] = distill_row(
            L[r], T[r], teacher_ids[r], teacher_values[r], int(lengths[r]), int(packed_width), float(grad_loss[r]), normalise)
    return out


def replay_gradient(logits, dtype, temperature, support_ids, lengths, packed_width, tokens, grad_token, grad_entries=None):
    """(gradient [B, V], magnitudes [B, V]) of the replay; zero rows where the replay gives no log-probability."""
    L = widen_logits(logits, dtype)
    B, V = L.shape
    T = np.asarray(temperature, np.float32).astype(np.float64)
    grad, mag = np.zeros((B, V)), np.zeros((B, V))
    for r in range(B):
        n = int(lengths[r])
        status, _, lp = replay_row(L[r], T[r], np.asarray(support_ids[r]), n, int(packed_width), int(tokens[r]))
        if status not in (ROW_OK, ROW_OUTSIDE):
            continue
        ids = np.asarray(support_ids[r][:n], np.int64)
        u = np.zeros(n) if grad_entries is None else np.asarray(grad_entries[r][:n], np.float64).copy()
        if status == ROW_OK:
            u[ids == int(tokens[r])] += float(grad_token[r])
        pi = np.exp(lp)
        grad[r, ids] = (u - pi * u.sum()) / T[r]
        mag[r, ids] = (np.abs(u) + pi * np.abs(u).sum()) / T[r]
    return grad, mag
