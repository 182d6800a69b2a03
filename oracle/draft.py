"""Verification of drafted tokens in plain numpy float64, one sequence at a
time, from the definitions of include/rlk_draft.h. The per-row statistics
(policy logprobs, support records) are inputs, as for the operator."""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import numpy as np

from .logp import decode_bf16


class Rows(NamedTuple):
    """Rows of logits and the forward call's statistics of them."""
    logits: np.ndarray                    # uint16 [n, >= vocab_real]
    temperature: np.ndarray               # float32 [n]
    policy: np.ndarray                    # float32 [n]
    lse_support: np.ndarray               # float32 [n]
    threshold: np.ndarray                 # float32 [n]
    status: np.ndarray                    # int32 [n]
    ref: Optional[np.ndarray] = None      # float32 [n]
    lse: Optional[np.ndarray] = None      # float32 [n]


def distribution(rows: Rows, i: int, vocab_real: int) -> np.ndarray:
    """The policy of row i over the real vocabulary (float64)."""
    x = decode_bf16(rows.logits[i, :vocab_real]).astype(np.float32)
    t = np.float32(rows.temperature[i])
    if t == 0:
        p = np.zeros(vocab_real)
        p[int(np.flatnonzero(x == x.max())[0])] = 1.0
        return p
    with np.errstate(over="ignore", invalid="ignore"):
        z = (x / t).astype(np.float64)
        p = np.exp(z - float(rows.lse_support[i]))
    return np.where(x >= rows.threshold[i], p, 0.0)


def usable(rows: Rows, i: int) -> bool:
    """Whether row i has a policy."""
    t = float(rows.temperature[i])
    if rows.status[i] < 0 or not 0 <= t < math.inf:
        return False
    return t == 0 or (math.isfinite(rows.lse_support[i]) and not math.isnan(rows.threshold[i]))


def verify(target: Rows, draft: Optional[Rows], vocab_real, start, token, accept_u, sample_u):
    """(tokens, accepted, policy, ref, margin): the outputs over the rows of the
    sequences, and per sequence the distance of the drawn token's borders from
    the random number, relative to the whole weight (inf where nothing is drawn)."""
    n = len(start) - 1
    rows = len(target.temperature)
    out = np.full(rows, -1, np.int64)
    accepted = np.full(n, -1, np.int32)
    policy, ref = np.zeros(rows), np.zeros(rows)
    margin = np.full(n, np.inf)
    for s in range(n):
        first, end = int(start[s]), int(start[s + 1])
        if not (0 <= first <= end <= len(token)):
            continue
        base, count = first + s, end - first
        k, wrong, q_row = 0, False, None
        while k < count:
            i, row = first + k, base + k
            lp, lq, q_row = float(target.policy[row]), 0.0, None
            wrong = not usable(target, row) or math.isnan(lp) or not 0 <= token[i] < vocab_real or not 0 <= accept_u[i] < 1
            if draft is not None:
                wrong = wrong or not usable(draft, i) or math.isnan(draft.policy[i])
                if draft.temperature[i] != 0:
                    lq, q_row = float(draft.policy[i]), i
            if wrong or lp == -math.inf:
                break
            ratio = math.inf if lp - lq > 700 else math.exp(lp - lq)
            if not accept_u[i] < ratio:
                break
            out[row], policy[row], ref[row] = token[i], target.policy[row], target.ref[row]
            k += 1
        accepted[s] = k
        row = base + k
        t = float(target.temperature[row])
        policy[row] = ref[row] = np.nan
        if wrong or not usable(target, row) or not 0 <= sample_u[s] < 1:
            continue
        r = distribution(target, row, vocab_real)
        if t == 0:
            out[row], policy[row], ref[row] = int(r.argmax()), 0.0, 0.0
            continue
        if k < count:
            q = np.zeros(vocab_real)
            if q_row is not None:
                q = distribution(draft, q_row, vocab_real)
            else:
                q[token[first + k]] = 1.0
            with np.errstate(invalid="ignore"):
                r = np.maximum(r - q, 0.0)
        sums = np.cumsum(r)
        if 0 < sums[-1] < math.inf:
            over = np.flatnonzero(sums > sample_u[s] * sums[-1])
            pick = int(over[0]) if over.size else int(np.flatnonzero(r > 0)[-1])
            near = np.abs(sums[max(0, pick - 1):pick + 1] - sample_u[s] * sums[-1])
            margin[s] = near.min() / sums[-1]
            z = float(np.float32(decode_bf16(target.logits[row, pick:pick + 1])[0]) / np.float32(t))
            out[row] = pick
            policy[row], ref[row] = z - float(target.lse_support[row]), z - float(target.lse[row])
        elif sums[-1] == 0 and k < count and target.policy[row] > -math.inf:
            out[row], policy[row], ref[row] = token[first + k], target.policy[row], target.ref[row]
    return out, accepted, policy, ref, margin
