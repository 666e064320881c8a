"""The embedding's gradient where a block sorts many entries over a wide range
of tokens (two passes, more entries than a warp holds in registers, several
rounds of the walk over the positions).  Whole numbers, whose sums are exact in
any order."""
import numpy as np
import pytest
import torch

from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu


def _tokens(kind, n, v, rng):
    tok = rng.integers(0, v, n)
    if kind == "low":                                   # frequent tokens have low numbers: most entries are one block's
        tok = np.minimum(np.exp(rng.random(n) * np.log(v + 1)).astype(np.int64), v) - 1
    elif kind == "one":                                 # one token and its neighbours
        tok = np.where(rng.random(n) < 0.6, v // 3, np.where(rng.random(n) < 0.8, v // 3 + rng.integers(-300, 300, n), tok))
    elif kind == "none":                                # most positions have no token
        tok = np.where(rng.random(n) < 0.9, -1 - rng.integers(0, 9, n), tok)
    elif kind == "last":
        tok = np.where(rng.random(n) < 0.5, v - 1, tok)
    return tok.astype(np.int32)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["even", "low", "one", "none", "last"])
@pytest.mark.parametrize("n,v,c", [(70001, 151936, 8), (140003, 300000, 16), (40000, 151936, 8)])
def test_exact_sums(n, v, c, kind, dtype, add):
    rng = np.random.default_rng(n + v)
    tok = torch.from_numpy(_tokens(kind, n, v, rng)).cuda()
    d = torch.from_numpy(rng.integers(-8, 9, (n, c)).astype(np.float32)).to(dtype).cuda()
    d[tok < 0] = float("nan")                           # not read
    desc = stp.embed_desc(n, v, c, stp.STP_BF16 if dtype == torch.bfloat16 else stp.STP_FP32, 0.5)
    ws = torch.full((stp.stp_embed_workspace_size(desc),), 255, dtype=torch.uint8, device="cuda")
    start = torch.arange(v * c, device="cuda", dtype=torch.float32).remainder_(997).view(v, c)
    got = start.clone() if add else torch.full((v, c), float("nan"), device="cuda")
    stp.stp_embed_bwd(desc, d, tok, add, got, ws)
    torch.cuda.synchronize()
    assert stp.stp_device_status(ws) == stp.STP_OK
    want = start.double() if add else torch.zeros(v, c, dtype=torch.float64, device="cuda")
    want.index_add_(0, tok[tok >= 0].long(), 0.5 * d[tok >= 0].double())
    assert float(want.abs().max()) < 2 ** 22 and torch.equal(got.double(), want)
