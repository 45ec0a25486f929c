"""Float64 CPU oracle of the verification of drafted tokens, over full rows and over captured supports.

TEST INFRASTRUCTURE, like the rest of this package. Request by request, position by position: draft x_j is
accepted while u_j q_j(x_j) < p_j(x_j); the next token wins the race argmax w_i / E_i over w = max(p - q, 0) at the
first refusal (p where that is zero everywhere), or p after the last draft. E_i = -ln v_i,
v_i = (2 (word >> 9) + 1) 2^-24, word i % 4 of the Philox4x32-10 block at (2^31 + i / 4, row, step).

``clear`` says whether every decision of a request clears float32 rounding: each accept by a relative margin, the
race by a winner whose weight, made smaller by the margin times p + q, still beats every other made larger by it.
"""
from __future__ import annotations

import dataclasses

import numpy as np

from .philox import philox4x32_10
from .sfc_oracle import ROW_BADPARAM, ROW_OK, ROW_OVERFLOW, widen_logits

MARGIN = 2.0 ** -15


@dataclasses.dataclass
class VerifyResult:
    accepted: np.ndarray  # int32 [B]
    tokens: np.ndarray  # int32 [B, D + 1]
    token_logprobs: np.ndarray  # float64 [B, D + 1]; NaN on requests that failed their checks
    row_status: np.ndarray  # int32 [B]
    clear: np.ndarray  # bool [B]


def waits(ids, row, seed, step):
    """E_i for token ids of one request."""
    ids = np.asarray(ids, np.uint64)
    quads, at = np.unique(ids >> np.uint64(2), return_inverse=True)
    n = quads.size
    ctr = [(quads + np.uint64(1 << 31)).astype(np.uint32), np.full(n, row, np.uint32),
           np.full(n, step & 0xFFFFFFFF, np.uint32), np.full(n, step >> 32, np.uint32)]
    block = np.stack(philox4x32_10(*ctr, np.uint32(seed & 0xFFFFFFFF), np.uint32(seed >> 32)))
    word = block[(ids & np.uint64(3)).astype(np.int64), at.reshape(-1)].astype(np.uint64)
    return -np.log((2.0 * (word >> np.uint64(9)).astype(np.float64) + 1.0) * 2.0 ** -24)


class Bad(Exception):
    def __init__(self, status):
        self.status = status


def _walk(n, drafted, uniforms, target, draft, row, seed, step):
    """One request: target(j) -> (ids, p), draft(j) -> {id: q} lookup function over an id array."""
    tokens, lps, clear = [], [], True
    while True:
        a = len(tokens)
        ids, p, lp = target(a)
        w, near = p, np.zeros_like(p)
        if a < n:
            x = int(drafted[a])
            q_at = draft(a, x)
            hit = np.flatnonzero(ids == x)
            px = float(p[hit[0]]) if hit.size else 0.0
            lpx = float(lp[hit[0]]) if hit.size else -np.inf
            if np.isnan(lpx) or lpx == np.inf:
                raise Bad(ROW_BADPARAM)
            left = float(uniforms[a]) * float(q_at(np.array([x]))[0])
            clear &= abs(left - px) > MARGIN * max(left, px) or left == px == 0.0
            if left < px:
                tokens.append(x)
                lps.append(lpx)
                continue
            q = q_at(ids)
            w, near = np.maximum(p - q, 0.0), MARGIN * (p + q)
            if not (w > 0).any():
                w, near = p, np.zeros_like(p)
        if (ids < 0).any() or np.isnan(lp).any() or np.isposinf(lp).any() or not (w > 0).any():
            raise Bad(ROW_BADPARAM)
        e = waits(ids, row, seed, step)
        ratio = w / e
        best = int(ids[ratio == ratio.max()].min())
        k = int(np.flatnonzero(ids == best)[0])
        others = np.delete((w + near) / e * (1 + MARGIN), k)
        clear &= others.size == 0 or (w[k] - near[k]) / e[k] > others.max()
        return a, tokens + [best], lps + [float(lp[k])], bool(clear)


def _collect(B, D, rows):
    out = VerifyResult(np.zeros(B, np.int32), np.full((B, D + 1), -1, np.int32), np.zeros((B, D + 1)), np.zeros(B, np.int32),
                       np.ones(B, bool))
    for b in range(B):
        try:
            out.accepted[b], tokens, lps, out.clear[b] = rows(b)
            out.tokens[b, :len(tokens)], out.token_logprobs[b, :len(lps)] = tokens, lps
        except Bad as e:
            out.row_status[b] = e.status
            out.token_logprobs[b] = np.nan
    return out


def distribution(l, T, greedy_t0):
    """(p, ln p) of one row of logits; T = 0 with greedy_t0: all on the lowest id among the largest."""
    if np.isnan(l).any() or np.isposinf(l).any() or not np.isfinite(l).any():
        raise Bad(ROW_BADPARAM)
    if T == 0.0 and greedy_t0:
        lp = np.full(l.shape, -np.inf)
        lp[int(np.argmax(l))] = 0.0
        return np.exp(lp), lp
    if not (np.isfinite(T) and T > 0.0):
        raise Bad(ROW_BADPARAM)
    z = l / T - (l / T).max()
    lp = z - np.log(np.exp(z).sum())
    return np.exp(lp), lp


def verify_drafts(target, draft, dtype, draft_tokens, uniforms, temperature, seed, step, draft_temperature=None, num_drafts=None,
                  greedy_t0=False, row_offset=0) -> VerifyResult:
    """target [B, D + 1, V], draft [B, D, V] or None: raw logits (bf16 bit patterns or float32)."""
    B, D = np.asarray(draft_tokens).shape
    V = target.shape[2]
    every = np.arange(V)
    Ts = np.asarray(temperature, np.float32).astype(np.float64)
    Td = Ts if draft_temperature is None else np.asarray(draft_temperature, np.float32).astype(np.float64)
    ok = lambda T: (np.isfinite(T) and T > 0) or (greedy_t0 and T == 0)

    def request(b):
        n = D if num_drafts is None else int(num_drafts[b])
        if n < 0 or n > D or not ok(Ts[b]) or (draft is not None and n > 0 and not ok(Td[b])):
            raise Bad(ROW_BADPARAM)

        def target_at(j):
            p, lp = distribution(widen_logits(target[b, j][None], dtype)[0], Ts[b], greedy_t0)
            return every, p, lp

        def draft_at(j, x):
            if x < 0 or x >= V:
                raise Bad(ROW_BADPARAM)
            if draft is None:
                return lambda ids: (ids == x).astype(np.float64)
            q, _ = distribution(widen_logits(draft[b, j][None], dtype)[0], Td[b], greedy_t0)
            return lambda ids: q[ids]

        return _walk(n, draft_tokens[b], uniforms[b], target_at, draft_at, (row_offset + b) & 0xFFFFFFFF, seed, step)

    return _collect(B, D, request)


def verify_supports(target_ids, target_lps, target_lengths, draft_ids, draft_lps, draft_lengths, draft_tokens, uniforms, seed,
                    step, num_drafts=None, row_offset=0) -> VerifyResult:
    B, D = np.asarray(draft_tokens).shape

    def request(b):
        n = D if num_drafts is None else int(num_drafts[b])
        if n < 0 or n > D:
            raise Bad(ROW_BADPARAM)

        def target_at(j):
            k = int(target_lengths[b, j])
            if k < 1 or k > target_ids.shape[2]:
                raise Bad(ROW_BADPARAM if k < 1 else ROW_OVERFLOW)
            lp = np.asarray(target_lps[b, j, :k], np.float64)
            return np.asarray(target_ids[b, j, :k], np.int64), np.exp(lp), lp

        def draft_at(j, x):
            k = 0 if draft_ids is None else int(draft_lengths[b, j])
            if k < 0 or x < 0 or (k and k > draft_ids.shape[2]):
                raise Bad(ROW_BADPARAM if k < 0 or x < 0 else ROW_OVERFLOW)
            if k == 0:
                return lambda ids: (np.asarray(ids) == x).astype(np.float64)
            q = {int(i): float(np.exp(np.float64(v))) for i, v in zip(draft_ids[b, j, :k], draft_lps[b, j, :k])}
            if not q.get(x, 0.0) < np.inf:
                raise Bad(ROW_BADPARAM)
            return lambda ids: np.array([q.get(int(i), 0.0) for i in ids])

        return _walk(n, draft_tokens[b], uniforms[b], target_at, draft_at, (row_offset + b) & 0xFFFFFFFF, seed, step)

    return _collect(B, D, request)
