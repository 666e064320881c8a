"""Gradients written over the logits that they are taken from, with one block
and with several blocks to a row: the bits of a gradient written elsewhere."""
import pytest
import torch

from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
DT = {stp.STP_BF16: torch.bfloat16, stp.STP_FP32: torch.float32}


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,v", [(3, 60001), (1, 151936), (700, 9001)])
def test_in_place(n, v, dtype):
    g = torch.Generator().manual_seed(n)
    z = (2 * torch.randn(n, v, generator=g)).to(DT[dtype]).cuda()
    t = torch.randint(0, v, (n,), generator=g).int().cuda()
    w, h = (torch.randn(n, generator=g).cuda() for _ in range(2))
    ids = torch.randint(0, v, (n, 200), generator=g).int().cuda()        # in every block's part
    tl = torch.randn(n, 200, generator=g).cuda()
    lp, ent, lse, loss = (torch.empty(n, device="cuda") for _ in range(4))
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    ds, dd = stp.stats_desc(n, v, 0, dtype), stp.distill_desc(n, v, 200, dtype)

    def stats(x, dz):
        stp.stp_token_stats_fwd(ds, x, t, lp, ent, lse, None, None, ws)
        stp.stp_token_stats_bwd(ds, x, t, lse, ent, w, h, dz)

    def two(x, dz):
        stp.stp_distill_fwd(dd, x, ids, tl, None, loss, lse, ws)
        stp.stp_distill_bwd(dd, x, ids, tl, None, lse, w, dz)

    def step(x, dz):
        stp.stp_distill_step(dd, x, ids, tl, None, w, loss, lse, dz, ws)

    for f in (stats, two, step):
        want, here = torch.full_like(z, float("nan")), z.clone()
        f(z, want)
        f(here, here)
        torch.cuda.synchronize()
        assert torch.isfinite(want).all() and torch.equal(want, here), f.__name__
