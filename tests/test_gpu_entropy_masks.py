"""Token statistics of rows that are masked with large finite values (the
type's lowest, -1e38) instead of -inf, beside ordinary logits: probability 0
for what is masked, and the same log-probability, entropy, top tokens and
gradient as with -inf there (oracle/token_loss.py in float64).

Tolerance, from the logits that carry weight alone (within 41 of the row's
maximum): the sum of V exponentials in chains of at most V / 256 + 96, each
2^x within 2^-22 and its argument within 2^-23 of 41 log2 e, and the float32
rounding of lse: e = (V / 256 + 96) 2^-24 + 2^-21 + 41 * 2^-22 + |lse| 2^-23.
Entropy sums p ln p, |ln p| < 41: 42 e.  A gradient's p carries 2 e relative;
the result is rounded once.
"""
import numpy as np
import pytest
import torch

from oracle import token_loss as OT
from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
DT = {stp.STP_BF16: torch.bfloat16, stp.STP_FP32: torch.float32}


def _masked(where, n, v, value, dtype, seed):
    """Ordinary logits, `value` in the masked columns; and the targets, in open columns."""
    rng = np.random.default_rng(seed)
    open_ = np.zeros((n, v), bool)
    if where == "before":
        open_[:, v // 2:] = True
    elif where == "after":
        open_[:, :max(8, v // 70)] = True
    elif where == "between":
        open_[:, :v // 3] = open_[:, -v // 3:] = True
    else:                       # a few open columns anywhere
        for r in range(n):
            open_[r, rng.choice(v, 8, replace=False)] = True
    z = torch.from_numpy((3 * rng.standard_normal((n, v))).astype(np.float32))
    z[torch.from_numpy(~open_)] = value
    targets = np.array([rng.choice(np.flatnonzero(o)) for o in open_], np.int32)
    return z.to(DT[dtype]).cuda(), targets


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("where", ["before", "after", "between", "few"])
@pytest.mark.parametrize("n,v,scale", [(2, 700, 1.0), (2, 40000, 1.0), (3, 20001, 0.5), (2, 40000, 2.0), (640, 2500, 1.0)])
@pytest.mark.parametrize("low", [-1e38, None])      # None: the type's lowest value
def test_finite_masks(n, v, scale, where, low, dtype):
    k, u = 5, torch.finfo(DT[dtype]).eps / 2
    z, targets = _masked(where, n, v, torch.finfo(DT[dtype]).min if low is None else low, dtype, seed=v + n)
    d = stp.stats_desc(n, v, k, dtype, scale)
    row = lambda: torch.full((n,), float("nan"), device="cuda")  # noqa: E731
    lp, ent, lse, top = row(), row(), row(), torch.full((n, k), float("nan"), device="cuda")
    ids, t = torch.full((n, k), -7, dtype=torch.int32, device="cuda"), torch.from_numpy(targets).cuda()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    stp.stp_token_stats_fwd(d, z, t, lp, ent, lse, ids, top, ws)
    rng = np.random.default_rng(1)
    g, h = (torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda() for _ in range(2))
    dz = torch.full_like(z, float("nan"))
    stp.stp_token_stats_bwd(d, z, t, lse, ent, g, h, dz)
    torch.cuda.synchronize()
    assert stp.stp_device_status(ws) == stp.STP_OK
    lp, ent, lse, ids, top, dz = (x.double().cpu().numpy() for x in (lp, ent, lse, ids, top, dz))
    zh = z.double().cpu().numpy()
    for r in range(n):
        w = OT.stats_row(zh[r], targets[r], k, scale)
        e = (v / 256 + 96) * 2.0 ** -24 + 2.0 ** -21 + 41 * 2.0 ** -22 + abs(w[2]) * 2.0 ** -23
        assert abs(lp[r] - w[0]) <= e and abs(lse[r] - w[2]) <= e
        assert abs(ent[r] - w[1]) <= 42 * e, (r, ent[r], w[1])
        assert ids[r].tolist() == w[3].tolist() and (np.abs(top[r] - w[4]) <= e).all()
        gr, hr = float(g[r]), float(h[r])
        want = OT.stats_grad_row(zh[r], targets[r], gr, hr, scale)
        p = np.exp(OT._log_softmax(zh[r] * scale)[0])
        tol = u * np.abs(want) + scale * p * (abs(gr) + 84 * abs(hr)) * 2 * e + 2.0 ** -22 * scale * abs(gr) + 1e-30
        assert (np.abs(dz[r] - want) <= tol).all(), r
