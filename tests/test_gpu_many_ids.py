"""Ids and targets outside the vocabulary where one block checks them all and
where every row checks its own: the device error word is set, and cleared by
the next call, wherever the bad one lies."""
import numpy as np
import pytest
import torch

from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,k", [(5, 3), (64, 64), (65, 64), (700, 64), (300, 256)])
@pytest.mark.parametrize("masked", [False, True])
def test_teacher_ids(n, k, masked):
    v = 900
    g = torch.Generator().manual_seed(n)
    z = torch.randn(n, v, generator=g).to(torch.bfloat16).cuda()
    ids = torch.randint(0, v, (n, k), generator=g).int().cuda()
    tl = torch.randn(n, k, generator=g).cuda()
    mask = torch.ones(n, dtype=torch.uint8, device="cuda") if masked else None
    loss, lse, w = (torch.ones(n, device="cuda") for _ in range(3))
    dz, ws = torch.empty_like(z), torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    d = stp.distill_desc(n, v, k)

    def status(how):
        if how == "step":
            stp.stp_distill_step(d, z, ids, tl, mask, w, loss, lse, dz, ws)
        else:
            stp.stp_distill_fwd(d, z, ids, tl, mask, loss, lse, ws)
        return stp.stp_device_status(ws)

    for how in ("fwd", "step"):
        assert status(how) == stp.STP_OK
        for at in ((0, 0), (n - 1, k - 1), (n // 2, k // 3)):
            keep = int(ids[at])
            ids[at] = v
            assert status(how) == stp.STP_EDEVICE
            if masked:
                mask[at[0]] = 0            # a row that is not read is not checked
                assert status(how) == stp.STP_OK
                mask[at[0]] = 1
            ids[at] = keep
            assert status(how) == stp.STP_OK


@pytest.mark.parametrize("n", [7, 4096, 4097, 9000])
def test_targets(n):
    v = 300
    z = torch.randn(n, v, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
    t = torch.from_numpy(np.random.default_rng(n).integers(-1, v, n).astype(np.int32)).cuda()
    out, ws = [torch.empty(n, device="cuda") for _ in range(3)], torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    d = stp.stats_desc(n, v)
    for bad in (None, 0, n - 1, n // 2, None):
        keep = t.clone()
        if bad is not None:
            t[bad] = v
        stp.stp_token_stats_fwd(d, z, t, *out, None, None, ws)
        assert stp.stp_device_status(ws) == (stp.STP_OK if bad is None else stp.STP_EDEVICE)
        assert torch.isnan(out[0]).sum() == (0 if bad is None else 1)
        t.copy_(keep)
