"""Token statistics of special rows side by side, each row with bounds from its
own logits (as in test_gpu_entropy_masks.py): a row at the ends of the type
does not widen what is asked of its neighbours."""
import numpy as np
import pytest
import torch

from oracle import token_loss as OT
from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
DT = {stp.STP_BF16: torch.bfloat16, stp.STP_FP32: torch.float32}


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,v", [(12, 5000), (640, 5000), (12, 60001)])
def test_special_rows(n, v, dtype):
    k, u = 32, torch.finfo(DT[dtype]).eps / 2
    rng = np.random.default_rng(n)
    z = torch.from_numpy((3 * rng.standard_normal((n, v))).astype(np.float32))
    targets = rng.integers(0, v, n).astype(np.int32)
    z[0] = 1.5                                         # all equal: the smallest ids
    z[1] = -float("inf")
    z[1, 4321] = -80.0                                 # one token alone
    targets[1] = 4321
    z[2] = torch.tensor([0.0, -0.0]).repeat(v)[:v]     # equal too
    z[3] = torch.arange(v) / 16
    z[4] = -torch.arange(v) / 16
    z[5, 8:16] = 30.0                                  # the largest all in one piece of the row
    z[6, ::2048] = 29.0                                # the largest all in one thread's strip
    z[7] = 3e38                                        # at the type's ends
    z[8] = -3e38
    z[9, 17:] = -float("inf")
    targets[9] = 3
    z[10] += 200.0
    z = z.to(DT[dtype])
    d = stp.stats_desc(n, v, k, dtype)
    row = lambda: torch.full((n,), float("nan"), device="cuda")  # noqa: E731
    lp, ent, lse, top = row(), row(), row(), torch.full((n, k), float("nan"), device="cuda")
    ids, t, zc = torch.full((n, k), -7, dtype=torch.int32, device="cuda"), torch.from_numpy(targets).cuda(), z.cuda()
    ws, dz = torch.empty(256, dtype=torch.uint8, device="cuda"), torch.full_like(zc, float("nan"))
    stp.stp_token_stats_fwd(d, zc, t, lp, ent, lse, ids, top, ws)
    g, h = (torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda() for _ in range(2))
    stp.stp_token_stats_bwd(d, zc, t, lse, ent, g, h, dz)
    torch.cuda.synchronize()
    assert stp.stp_device_status(ws) == stp.STP_OK
    lp, ent, lse, ids, top, dz = (x.double().cpu().numpy() for x in (lp, ent, lse, ids, top, dz))
    zh = z.double().numpy()
    for r in range(n):
        w = OT.stats_row(zh[r], targets[r], k)
        far = abs(w[0]) * 2.0 ** -22                   # of a log-probability far from the maximum
        e = (v / 256 + 96) * 2.0 ** -24 + 2.0 ** -21 + 41 * 2.0 ** -22
        assert abs(lp[r] - w[0]) <= e + far, r
        assert abs(lse[r] - w[2]) <= e + abs(w[2]) * 2.0 ** -23, r
        assert abs(ent[r] - w[1]) <= 42 * e, (r, ent[r], w[1])
        assert ids[r].tolist() == w[3].tolist(), r
        live = np.isfinite(w[4])
        assert np.array_equal(live, np.isfinite(top[r]))
        assert (np.abs(top[r][live] - w[4][live]) <= e + np.abs(w[4][live]) * 2.0 ** -22).all(), r
        if abs(w[2]) > 1e5:
            continue                                   # the separate backward has lse alone
        e += abs(w[2]) * 2.0 ** -23
        gr, hr = float(g[r]), float(h[r])
        want = OT.stats_grad_row(zh[r], targets[r], gr, hr)
        p = np.exp(OT._log_softmax(zh[r])[0])
        tol = u * np.abs(want) + p * (abs(gr) + 84 * abs(hr)) * 2 * e + 2.0 ** -22 * abs(gr) + 1e-30
        assert (np.abs(dz[r] - want) <= tol).all(), r
