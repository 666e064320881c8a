"""The embedding's gradient added to a table that holds numbers below
float32's smallest normal one (stp_embed_bwd, accumulate): they count like any
other.  The values are whole multiples of 2^-149 or 2^-126 with few bits, so
that every sum is exact."""
import numpy as np
import pytest
import torch

from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
DT = {stp.STP_BF16: torch.bfloat16, stp.STP_FP32: torch.float32}


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,v,c", [(5, 40, 8), (300, 90, 264), (5000, 7, 1032)])    # tokens that occur once, some and many times
def test_small_sums(n, v, c, dtype, add):
    rng = np.random.default_rng(n)
    tok = rng.integers(0, v, n).astype(np.int32)
    step = 2.0 ** -133 if dtype == stp.STP_BF16 else 2.0 ** -149                     # the type's smallest number
    d = torch.from_numpy(rng.integers(-1, 2, (n, c)) * step).to(DT[dtype])
    start = torch.from_numpy(rng.integers(-1000, 1001, (v, c)) * 2.0 ** -149).float()
    start[0] = 2.0 ** -126                                                            # the sum is below it, or above
    desc, t = stp.embed_desc(n, v, c, dtype), torch.from_numpy(tok)
    grad, ws = start.cuda().clone(), torch.empty(stp.stp_embed_workspace_size(desc), dtype=torch.uint8, device="cuda")
    stp.stp_embed_bwd(desc, d.cuda(), t.cuda(), add, grad, ws)
    torch.cuda.synchronize()
    assert stp.stp_device_status(ws) == stp.STP_OK
    want = start.double() if add else torch.zeros(v, c, dtype=torch.float64)
    want.index_add_(0, t.long(), d.double())
    assert torch.equal(want.float().double(), want)
    assert torch.equal(grad.double().cpu(), want)


@pytest.mark.parametrize("n", [3, 200])
def test_sums_that_cancel(n):
    # what is left of a normal number is below the smallest normal one
    start = torch.full((1, 8), 2.0 ** -126)
    d = torch.zeros(n, 8)
    d[n // 2] = -(2.0 ** -126) + 2.0 ** -140
    desc = stp.embed_desc(n, 1, 8, stp.STP_FP32)
    grad, ws = start.cuda(), torch.empty(stp.stp_embed_workspace_size(desc), dtype=torch.uint8, device="cuda")
    stp.stp_embed_bwd(desc, d.cuda(), torch.zeros(n, dtype=torch.int32, device="cuda"), True, grad, ws)
    torch.cuda.synchronize()
    assert torch.equal(grad.cpu(), torch.full((1, 8), 2.0 ** -140))
