"""Windowed tree attention on rows of many tiles: lists longer than twice the
ring of visibility words, odd head groups, and rows of more than 128 tiles,
which the classification walks in several turns.

The reference is dense float64 attention under the definition
  j <= i, subtree_end[j] >= i, position[i] - position[j] < window or position[j] < n_sink,
computed a strip of queries at a time.  Tolerance: what rounding P, dS and the
stored O once to bf16 does at most (u = 2^-8), and float32 sums of n terms,
n / 2 * 2^-24 of the sums of absolute values; n is the number of keys that a
query sees, or of queries and heads that see a key, 1024 at least.
"""
import numpy as np
import pytest
import torch

from sft_trie_build_gb300 import stp
from test_gpu_window import Run, _forest

pytestmark = pytest.mark.gpu


def _see(se, pos, i, window, sinks):
    j = torch.arange(len(se), device=se.device)
    near = (pos[i][:, None] - pos[None] < window) | (pos[None] < sinks)
    return (j[None] <= i[:, None]) & (se[None] >= i[:, None]) & near


def _dense(r, scale):
    q, k, v, do = (x.double() for x in (r.q, r.k, r.v, r.do))
    R, T, hq, _ = q.shape
    G = hq // k.shape[2]
    out = {x: torch.zeros_like(q) for x in ("o", "dq", "o_tol", "dq_tol")}
    out.update({x: torch.zeros_like(k) for x in ("dk", "dv", "dk_tol", "dv_tol")})
    out["lse"] = torch.zeros(R, hq, T, dtype=torch.float64, device="cuda")
    n, seen = 1024, torch.zeros(R, T, dtype=torch.int64, device="cuda")
    for row in range(R):
        for a in range(0, T, 1280):
            i = torch.arange(a, min(T, a + 1280), device="cuda")
            m = _see(r.se[row].long(), r.pos[row].long(), i, r.window, r.sinks)
            n = max(n, int(m.sum(1).max()))
            seen[row] += m.sum(0)
            for h in range(hq):
                g = h // G
                kk, vv, d, qq = k[row, :, g], v[row, :, g], do[row, i, h], q[row, i, h]
                s = (scale * qq @ kk.T).masked_fill_(~m, float("-inf"))
                lse = torch.logsumexp(s, 1, keepdim=True)
                p = torch.exp(s - lse)
                o = p @ vv
                o_tol = p @ vv.abs() + o.abs()
                ds = p * (d @ vv.T - (d * o).sum(1, keepdim=True))
                ds_tol = ds.abs() + p * (d.abs() * o_tol).sum(1, keepdim=True)
                out["o"][row, i, h], out["o_tol"][row, i, h], out["lse"][row, h, i] = o, o_tol, lse[:, 0]
                out["dq"][row, i, h], out["dq_tol"][row, i, h] = scale * ds @ kk, scale * ds_tol @ kk.abs()
                out["dk"][row, :, g] += scale * ds.T @ qq
                out["dk_tol"][row, :, g] += scale * ds_tol.T @ qq.abs()
                out["dv"][row, :, g] += p.T @ d
                out["dv_tol"][row, :, g] += p.T @ d.abs()
    for x in ("dq", "dk", "dv"):
        out[x + "_tol"] += out[x].abs()
    return out, max(n, int(seen.max()) * G) / 2 * 2.0 ** -24


def _sequence(T):
    return np.full((1, T), T - 1, np.int32), np.arange(T, dtype=np.int32)[None]


def _trees(T, seed, n_roots, lo, hi):
    plan = _forest(seed, T, n_roots=n_roots, len_lo=lo, len_hi=hi)
    return plan.subtree_end[:1], plan.position_ids[:1]


@pytest.mark.parametrize("hq,hkv,window,sinks,rows", [
    (1, 1, 1400, 0, (_sequence, 2560)),                   # one head of a pair, 12 tiles a list
    (3, 1, 2 ** 31 - 1, 0, (_sequence, 2304)),            # a pair and a single head, 18 tiles
    (2, 1, 1100, 300, (_sequence, 2560)),
    (4, 2, 700, 40, (_trees, 4096, 31, 3, 100, 1000)),
    (1, 1, 1500, 130, (_sequence, 16640)),                # 130 tiles
    (2, 1, 900, 20, (_trees, 20480, 32, 6, 50, 4000)),
])
def test_long_lists_and_rows(hq, hkv, window, sinks, rows):
    se, pos = rows[0](*rows[1:])
    r = Run(se, pos, hq, hkv, 128, stp.STP_BF16, window, sinks, seed=hq)
    r.step()
    got = r.outputs()
    want, work = _dense(r, r.desc.c().scale)
    assert np.abs(got["lse"] - want["lse"].cpu().numpy()).max() <= 32 * work
    for x in ("o", "dq", "dk", "dv"):
        off = np.abs(got[x] - want[x].cpu().numpy()) - (2.0 ** -8 + work) * want[x + "_tol"].cpu().numpy()
        assert off.max() <= 1e-6, (x, off.max())
    # the classes: what is visible lies in listed tiles, what is FULL is visible
    c, n = r.classes()[0], se.shape[1] // 128
    any_, all_ = np.zeros((n, n), bool), np.zeros((n, n), bool)
    for t in range(n):
        m = _see(r.se[0].long(), r.pos[0].long(), torch.arange(t * 128, t * 128 + 128, device="cuda"), window, sinks)
        m = m.view(128, n, 128)
        any_[t], all_[t] = m.any(2).any(0).cpu().numpy(), m.all(2).all(0).cpu().numpy()
    assert not (any_ & (c == 0)).any() and not (~all_ & (c == 2)).any()
    assert (c != 0).sum() == r.pairs
    lists = (c != 0).sum(1)
    assert lists.max() > 8 or window < 1000
