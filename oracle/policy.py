"""Float64 CPU oracle of the log-probabilities over a whole vocabulary, the policy loss, and gradient clipping.

TEST INFRASTRUCTURE, like the rest of this package. Row by row from the definitions (z = l / T): log-probabilities by the
log-softmax, the entropy by its sum, the alternatives by a stable sort, gradients from the Jacobian of the log-softmax and
dH = -sum (ln p + 1) dp, not from the library's arrangement of the sums.
"""
from __future__ import annotations

import dataclasses
import math

import numpy as np

from .distill import _log_softmax
from .sfc_oracle import ROW_BADPARAM, ROW_OK, widen_logits


@dataclasses.dataclass
class LogprobsResult:
    logprobs: np.ndarray  # float64 [B, M]
    entropy: np.ndarray  # float64 [B]
    top_ids: np.ndarray  # int32 [B, K]
    top_logprobs: np.ndarray  # float64 [B, K]
    row_status: np.ndarray  # int32 [B]
    far: np.ndarray  # float64 [B, V]: |z - max z| (infinite where masked)
    ln_mass: np.ndarray  # float64 [B]: ln sum exp(z - max z)
    spread: np.ndarray  # float64 [B]: sum p (z - max z)^2


@dataclasses.dataclass
class GradResult:
    grad: np.ndarray  # float64 [B, V]
    grad_scale: np.ndarray  # float64 [B, V]: the sum of the magnitudes that an entry is a difference of


def row_ok(l, T):
    return np.isfinite(T) and T > 0.0 and not np.isnan(l).any() and not np.isposinf(l).any() and np.isfinite(l).any()


def row_entropy(ln_p):
    p = np.exp(ln_p)
    return -float(np.sum(p[p > 0] * ln_p[p > 0]))


def token_logprobs(logits, dtype, temperature, tokens, top=0) -> LogprobsResult:
    L = widen_logits(logits, dtype)
    B, V = L.shape
    tokens = np.asarray(tokens).reshape(B, -1)
    T = np.asarray(temperature, np.float32).astype(np.float64)
    nan = lambda *shape: np.full(shape, np.nan)
    out = LogprobsResult(nan(*tokens.shape), nan(B), np.full((B, top), -1, np.int32), nan(B, top), np.full(B, ROW_BADPARAM, np.int32),
                         np.zeros((B, V)), np.zeros(B), np.zeros(B))
    for r in range(B):
        if not row_ok(L[r], T[r]) or (tokens[r] < -1).any() or (tokens[r] >= V).any():
            continue
        out.row_status[r] = ROW_OK
        z = L[r] / T[r]
        ln_p, out.far[r] = _log_softmax(z), z.max() - z
        p = np.exp(ln_p)
        out.ln_mass[r], out.spread[r] = -ln_p.max(), np.sum(p[p > 0] * out.far[r][p > 0] ** 2)
        out.logprobs[r] = np.where(tokens[r] >= 0, ln_p[np.maximum(tokens[r], 0)], 0.0)
        out.entropy[r] = row_entropy(ln_p)
        order = np.argsort(-L[r], kind="stable")[:top]
        order = order[np.isfinite(L[r][order])]
        out.top_ids[r, :len(order)], out.top_logprobs[r] = order, -np.inf
        out.top_logprobs[r, :len(order)] = ln_p[order]
    return out


def _gradient_row(ln_p, given, T):
    """(gradient, magnitudes) of sum_i g_i ln p_i + h H over one row; given = ([(id, g_i)], h)."""
    entries, h = given
    p = np.exp(ln_p)
    grad, mag = np.zeros(len(p)), np.zeros(len(p))
    for i, g in entries:
        if i < 0 or i >= len(p) or not np.isfinite(ln_p[i]):
            continue
        grad -= g * p
        mag += abs(g) * p
        grad[i] += g
        mag[i] += abs(g)
    if h != 0.0:
        # dH = -sum_k (ln p_k + 1) dp_k with dp_k / dz_j = p_k (delta_jk - p_j)
        on = p > 0
        inner = np.zeros(len(p))
        inner[on] = p[on] * (ln_p[on] + 1)
        grad += h * -(inner - p * inner.sum())
        mag[on] += abs(h) * p[on] * (np.abs(ln_p[on]) + row_entropy(ln_p) + 2 + np.sum(p[on] * ln_p[on] ** 2) / 8)
    return grad / T, mag / T


def token_logprobs_gradient(logits, dtype, temperature, tokens, grad_logprobs, grad_entropy=None) -> GradResult:
    L = widen_logits(logits, dtype)
    B, V = L.shape
    tokens, up = np.asarray(tokens).reshape(B, -1), np.asarray(grad_logprobs, np.float64).reshape(B, -1)
    T = np.asarray(temperature, np.float32).astype(np.float64)
    out = GradResult(np.zeros((B, V)), np.zeros((B, V)))
    for r in range(B):
        if row_ok(L[r], T[r]) and not (tokens[r] < -1).any() and not (tokens[r] >= V).any():
            h = 0.0 if grad_entropy is None else float(grad_entropy[r])
            out.grad[r], out.grad_scale[r] = _gradient_row(_log_softmax(L[r] / T[r]), (list(zip(tokens[r], up[r])), h), T[r])
    return out


@dataclasses.dataclass
class PolicyResult:
    loss: np.ndarray  # float64 [B]
    logprobs: np.ndarray  # float64 [B]
    entropy: np.ndarray  # float64 [B]
    slope: np.ndarray  # float64 [B]: dloss / dlogprob
    grad: np.ndarray  # float64 [B, V]
    grad_scale: np.ndarray  # float64 [B, V]
    row_status: np.ndarray  # int32 [B]


def policy_loss(logits, dtype, temperature, tokens, advantages, grad_loss, old_logprobs=None, clip_low=0.2, clip_high=0.2,
                entropy_weight=0.0) -> PolicyResult:
    L = widen_logits(logits, dtype)
    B, V = L.shape
    T = np.asarray(temperature, np.float32).astype(np.float64)
    zeros = lambda *shape: np.zeros(shape)
    out = PolicyResult(zeros(B), zeros(B), zeros(B), zeros(B), zeros(B, V), zeros(B, V), np.zeros(B, np.int32))
    for r in range(B):
        t, A = int(tokens[r]), float(advantages[r])
        old = None if old_logprobs is None else float(old_logprobs[r])
        ok = np.isfinite(T[r]) and T[r] > 0 and -1 <= t < V and np.isfinite(A) and (old is None or np.isfinite(old))
        if ok and t >= 0:
            ok = row_ok(L[r], T[r])
        if not ok:
            out.row_status[r] = ROW_BADPARAM
            out.loss[r] = out.logprobs[r] = out.entropy[r] = np.nan
            continue
        if t < 0:
            continue
        ln_p = _log_softmax(L[r] / T[r])
        lp, H = float(ln_p[t]), row_entropy(ln_p)
        if old is None:
            gain = 0.0 if A == 0 else A * lp
            slope = -A if np.isfinite(lp) else 0.0
        else:
            rho = math.exp(min(lp - old, 700.0))
            clamped = min(max(rho, 1 - clip_low), 1 + clip_high)
            gain = min(rho * A, clamped * A)
            slope = -rho * A if rho * A <= clamped * A else 0.0
        out.logprobs[r], out.entropy[r], out.slope[r] = lp, H, slope
        out.loss[r] = -gain - entropy_weight * H
        up = float(grad_loss[r])
        out.grad[r], out.grad_scale[r] = _gradient_row(ln_p, ([(t, slope * up)], -entropy_weight * up), T[r])
    return out


def grad_norm(grads):
    """The global norm of float64 arrays."""
    with np.errstate(over="ignore", invalid="ignore"):
        return math.sqrt(float(np.sum([np.sum(np.square(np.asarray(g, np.float64))) for g in grads])))


def clip_scale(norm, max_norm):
    if max_norm == math.inf:
        return 1.0
    ratio = max_norm / (norm + 1e-6) if norm != math.inf else 0.0
    return 1.0 if ratio >= 1.0 else ratio
