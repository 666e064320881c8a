"""Oracle: tree attention with a sliding window and visible first tokens, float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The visible keys of a query are its own path from the root (RowTree.visible,
from the packer's parent pointers); of the n tokens of that path the query
sees the last ``window`` and the first ``n_sink``.  Neither subtree_end nor
position ids are used, so a packed row is checked against what the sequence
alone would see.  A pad sees itself.
"""
from __future__ import annotations

import numpy as np

from .attn import RowTree
from .pack import Plan


def visible(rt: RowTree, i: int, window: int, n_sink: int) -> np.ndarray:
    keys = rt.visible(i)
    k = np.arange(len(keys))
    return keys[(k >= len(keys) - window) | (k < n_sink)]


def mask(plan: Plan, window: int, n_sink: int) -> np.ndarray:
    """bool [R, T, T]: entry (i, j) is True iff query i sees key j."""
    m = np.zeros((plan.n_rows, plan.row_len, plan.row_len), bool)
    for r in range(plan.n_rows):
        rt = RowTree(plan, r)
        for i in range(plan.row_len):
            m[r, i, visible(rt, i, window, n_sink)] = True
    return m


def attention(m: np.ndarray, q, k, v, scale: float, do=None) -> dict:
    """Dense attention under the mask m [R, T, T]; q, do [R, T, Hq, D], k, v
    [R, T, Hkv, D] -> o, lse [R, Hq, T] and, with do, dq, dk, dv; also the
    largest errors (o_tol, dq_tol, ...) that rounding P, dS and O once to a
    type of relative half step u can cause, per unit of u."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    R, T, Hq, D = q.shape
    G = Hq // k.shape[2]
    out = {x: np.zeros(q.shape) for x in ("o", "dq", "o_tol", "dq_tol")}
    out.update({x: np.zeros(k.shape) for x in ("dk", "dv", "dk_tol", "dv_tol")})
    out["lse"] = np.zeros((R, Hq, T))
    for r in range(R):
        for h in range(Hq):
            g = h // G
            kk, vv = k[r, :, g], v[r, :, g]
            s = np.where(m[r], scale * q[r, :, h] @ kk.T, -np.inf)
            mx = s.max(1, keepdims=True)
            e = np.exp(s - mx)
            z = e.sum(1, keepdims=True)
            p = e / z
            o = p @ vv
            o_tol = p @ np.abs(vv) + np.abs(o)
            out["o"][r, :, h], out["o_tol"][r, :, h], out["lse"][r, h] = o, o_tol, (mx + np.log(z))[:, 0]
            if do is None:
                continue
            d = np.asarray(do, np.float64)[r, :, h]
            ds = p * (d @ vv.T - (d * o).sum(1, keepdims=True))
            ds_tol = np.abs(ds) + p * (np.abs(d) * o_tol).sum(1, keepdims=True)
            out["dq"][r, :, h], out["dq_tol"][r, :, h] = scale * ds @ kk, scale * ds_tol @ np.abs(kk)
            out["dk"][r, :, g] += scale * ds.T @ q[r, :, h]
            out["dk_tol"][r, :, g] += scale * ds_tol.T @ np.abs(q[r, :, h])
            out["dv"][r, :, g] += p.T @ d
            out["dv_tol"][r, :, g] += p.T @ np.abs(d)
    for x in ("dq", "dk", "dv"):
        out[x + "_tol"] += np.abs(out[x])
    return out
