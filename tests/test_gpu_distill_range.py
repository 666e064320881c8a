"""The one-launch distillation step on rows whose logits are large: all of the
type's lowest value, or offsets that a float32 log-sum-exp cannot carry.  Loss
and gradient follow the differences to the row's maximum, so that they are
those of the same row near zero.

Tolerance: e of the differences that carry weight (within 41 of the maximum),
(V / 256 + 96) 2^-24 + 2^-21 + 41 * 2^-22 relative on p; loss and q as in
test_gpu_token_loss.py, with the differences in place of the logits: 2^-22 of
the largest one among the listed ids on the loss.
"""
import numpy as np
import pytest
import torch

from oracle import token_loss as OT
from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
DT = {stp.STP_BF16: torch.bfloat16, stp.STP_FP32: torch.float32}


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("scale", [1.0, 1.5, 0.25])
@pytest.mark.parametrize("n,v", [(6, 700), (6, 40000), (640, 1001)])
def test_step_follows_differences(n, v, scale, dtype):
    dt, k = DT[dtype], 9
    u = torch.finfo(dt).eps / 2
    rng = np.random.default_rng(v)
    z = torch.from_numpy((2 * rng.standard_normal((n, v))).astype(np.float32))
    z[0] = torch.finfo(dt).min                     # all alike
    z[1] = -torch.finfo(dt).max / 8
    z[2] = 3e37
    z[3] += 40000.0                                # p from a rounded lse: off by 2^-9 and more
    z[4] -= 3e6
    z[5, 10:] = torch.finfo(dt).min
    z = z.to(dt)
    ids = np.stack([rng.choice(min(v, 10) if r == 5 else v, k, replace=False) for r in range(n)]).astype(np.int32)
    tl = (2 * rng.standard_normal((n, k))).astype(np.float32)
    d = stp.distill_desc(n, v, k, dtype, scale)
    g = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    loss, lse = torch.full((n,), float("nan"), device="cuda"), torch.full((n,), float("nan"), device="cuda")
    zc, dz = z.cuda(), torch.full_like(z, float("nan"), device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    stp.stp_distill_step(d, zc, torch.from_numpy(ids).cuda(), torch.from_numpy(tl).cuda(), None, g, loss, lse, dz, ws)
    torch.cuda.synchronize()
    assert stp.stp_device_status(ws) == stp.STP_OK
    e = (v / 256 + 96) * 2.0 ** -24 + 2.0 ** -21 + 41 * 2.0 ** -22
    zh, dz = z.double().numpy(), dz.double().cpu().numpy()
    for r in range(n):
        want, wl = OT.distill_row(zh[r], ids[r], tl[r], scale)
        a, far = np.abs(tl[r]).max() * scale, np.abs(zh[r][ids[r]] - zh[r].max()).max() * scale
        assert abs(float(loss[r]) - want) <= (2 * e + (k + 8) * 2.0 ** -24 * 41 + a * 2.0 ** -21 + far * 2.0 ** -22), r
        with np.errstate(over="ignore"):           # beyond float32, lse is infinite
            assert float(lse[r]) == np.float32(wl) or abs(float(lse[r]) - wl) <= e + abs(wl) * 2.0 ** -22
        want, gn = OT.distill_grad_row(zh[r], ids[r], tl[r], float(g[r]), scale), abs(float(g[r])) * scale
        p, q = np.exp(OT._log_softmax(zh[r] * scale)[0]), np.zeros(v)
        np.add.at(q, ids[r], OT._teacher(ids[r], tl[r], scale)[1])
        tol = u * np.abs(want) + gn * (2 * e * p + ((k + 16) * 2.0 ** -24 + a * 2.0 ** -21) * q) + 1e-30
        assert (np.abs(dz[r] - want) <= tol).all(), r
