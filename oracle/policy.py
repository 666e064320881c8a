"""Oracle: clipped policy loss with a KL and an entropy term on one row of
logits, and its gradient, float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

With lp the target's log-probability, H the entropy, r = exp(lp - old) and
k = exp(ref - lp) - (ref - lp) - 1:

    loss = -min(r A, clip(r, 1 - low, 1 + high) A) + kl_coef k - entropy_coef H
"""
from __future__ import annotations

import numpy as np

from oracle import token_loss as OT


def terms(lp, ent, old, ref, adv, low, high, kl_coef, entropy_coef):
    """(loss, kl, d loss / d lp) of one row; ref None: no KL term."""
    r = np.exp(lp - old)
    edge = 1 + high if adv >= 0 else 1 - low
    out = r > edge if adv >= 0 else r < edge
    loss = -adv * (edge if out else r) - entropy_coef * ent
    g = 0.0 if out else -adv * r
    kl = 0.0
    if ref is not None:
        x = ref - lp
        kl = np.expm1(x) - x
        if kl_coef:
            loss += kl_coef * kl
            g -= kl_coef * np.expm1(x)
    return loss, kl, g


def row(logits, target, old, ref, adv, low, high, kl_coef, entropy_coef, scale=1.0):
    """(loss, logprob, entropy, lse, kl, gradient by the logits) of one row."""
    lp, ent, lse, _, _ = OT.stats_row(logits, target, 0, scale)
    loss, kl, g = terms(lp, ent, old, ref, adv, low, high, kl_coef, entropy_coef)
    if lp == -np.inf:
        return loss, lp, ent, lse, kl, np.zeros(len(logits))
    return loss, lp, ent, lse, kl, OT.stats_grad_row(logits, target, g, -entropy_coef, scale)
