"""The gradient of token statistics with large weights of the entropy beside
masked logits: what has probability 0 has a gradient of 0
(stp_token_stats_bwd).  Bounds as in tests/test_gpu_entropy_masks.py."""
import numpy as np
import pytest
import torch

from oracle import token_loss as OT
from sft_trie_build_gb300 import stp
from test_gpu_entropy_masks import DT, _masked

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low", [-float("inf"), None])                # None: the type's lowest value
@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,v", [(4, 701), (2, 40001)])               # one and several blocks to a row
def test_masked_logits_have_no_gradient(n, v, dtype, low):
    z, targets = _masked("between", n, v, torch.finfo(DT[dtype]).min if low is None else low, dtype, seed=v)
    d = stp.stats_desc(n, v, 0, dtype)
    lp, ent, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(3))
    t, ws = torch.from_numpy(targets).cuda(), torch.empty(256, dtype=torch.uint8, device="cuda")
    stp.stp_token_stats_fwd(d, z, t, lp, ent, lse, None, None, ws)
    g, h = torch.full((n,), 0.5, device="cuda"), torch.full((n,), 1e9, device="cuda")
    dz = torch.full_like(z, float("nan"))
    stp.stp_token_stats_bwd(d, z, t, lse, ent, g, h, dz)
    torch.cuda.synchronize()
    assert stp.stp_device_status(ws) == stp.STP_OK
    zh, got, u = z.double().cpu().numpy(), dz.double().cpu().numpy(), torch.finfo(DT[dtype]).eps / 2
    masked = zh < -1e30
    assert masked.any() and (got[masked] == 0).all()
    for r in range(n):
        _, _, want_lse, _, _ = OT.stats_row(zh[r], targets[r])
        e = (v / 256 + 96) * 2.0 ** -24 + 2.0 ** -21 + 41 * 2.0 ** -22 + abs(want_lse) * 2.0 ** -23
        p = np.exp(OT._log_softmax(zh[r])[0])
        want = OT.stats_grad_row(zh[r], targets[r], 0.5, 1e9)
        tol = u * np.abs(want) + p * (0.5 + 84e9) * 2 * e + 2.0 ** -23 + 1e-30
        assert (np.abs(got[r] - want) <= tol).all(), r
