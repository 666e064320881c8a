"""Oracle: statistics of rows of logits and distillation from a teacher's top
logits, with their gradients, float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

With z = scale * logits of a row and p = softmax(z):

    logprob = ln p_target,  entropy = -sum p ln p,
    alternatives: the top_k largest logits, descending, ties to the smaller id
    distillation: q = softmax(scale * teacher_logits) over the listed ids,
                  loss = sum_k q_k (ln q_k - ln p_{id_k})
"""
from __future__ import annotations

import numpy as np


def _log_softmax(z: np.ndarray):
    """(z - ln sum exp z, ln sum exp z); the difference to the maximum comes
    first, so that a row of one huge value stays an even distribution."""
    mx = z.max()
    if mx == -np.inf:
        return np.full_like(z, -np.inf), -np.inf
    ls = np.log(np.exp(z - mx).sum())
    return (z - mx) - ls, mx + ls


def stats_row(logits, target: int, top_k: int = 0, scale: float = 1.0):
    """(logprob, entropy, lse, ids [top_k], logprobs [top_k]) of one row; ids -1 where none is left."""
    raw = np.asarray(logits, np.float64)
    lp, lse = _log_softmax(raw * scale)
    live = lp > -np.inf
    ent = float(-(np.exp(lp[live]) * lp[live]).sum())
    order = np.lexsort((np.arange(len(raw)), -raw))
    order = order[raw[order] > -np.inf][:top_k]
    ids = np.full(top_k, -1, np.int32)
    top = np.full(top_k, -np.inf)
    ids[:len(order)], top[:len(order)] = order, lp[order]
    return lp[target], ent, lse, ids, top


def stats_grad_row(logits, target: int, g_logprob: float, g_entropy: float, scale: float = 1.0) -> np.ndarray:
    """Gradient of g_logprob * logprob + g_entropy * entropy."""
    lp, _ = _log_softmax(np.asarray(logits, np.float64) * scale)
    p = np.exp(lp)
    safe = np.where(p > 0, lp, 0.0)
    ent = -(p * safe).sum()
    hot = np.arange(len(lp)) == target
    return scale * (g_logprob * (hot - p) - g_entropy * p * (safe + ent))


def _teacher(ids, teacher_logits, scale):
    ids = np.asarray(ids)
    a = np.asarray(teacher_logits, np.float64) * scale
    on = (ids >= 0) & (a > -np.inf)
    q = np.zeros(len(ids))
    if on.any():
        q[on] = np.exp(_log_softmax(a[on])[0])
    return ids, q, on


def distill_row(logits, ids, teacher_logits, scale: float = 1.0):
    """(loss, lse) of one row; (0, 0) where no id is listed."""
    ids, q, on = _teacher(ids, teacher_logits, scale)
    if not on.any():
        return 0.0, 0.0
    lp, lse = _log_softmax(np.asarray(logits, np.float64) * scale)
    on = on & (q > 0)
    return float((q[on] * (np.log(q[on]) - lp[ids[on]])).sum()), lse


def distill_grad_row(logits, ids, teacher_logits, g: float, scale: float = 1.0) -> np.ndarray:
    """Gradient of g * loss."""
    ids, q, on = _teacher(ids, teacher_logits, scale)
    if not on.any():
        return np.zeros(len(logits))
    d = np.exp(_log_softmax(np.asarray(logits, np.float64) * scale)[0])
    np.subtract.at(d, ids[on], q[on])
    return g * scale * d
