"""Embedding and its gradient on the GPU (stp_embed_*) against the float64
oracle (oracle/embed.py).

Tolerance.  A vector is a product rounded to float32, then once to its type:
(2^-24 + u) relative.  A gradient adds m rows of d_out in float32, in chains of at most m, then
scales them and perhaps adds them to what was there: (m + 2) 2^-24 of the sum
of magnitudes, and 2^-24 of the result.
"""
import numpy as np
import pytest
import torch

from oracle import embed as OE
from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
DT = {stp.STP_BF16: torch.bfloat16, stp.STP_FP32: torch.float32}
NAN = float("nan")


def _tokens(kind, n, v, rng):
    if kind == "one":                                   # pads: one token many times
        t = np.zeros(n, np.int64) + v // 2
    elif kind == "few":
        t = rng.integers(0, min(v, 3), n)
    elif kind == "runs":                                # ends of tokens on, before and behind the ends of pieces
        t = np.repeat(np.arange(n), rng.choice([1, 31, 32, 33, 64, 65], n))[:n] % v
        t = rng.permutation(t)
    else:
        t = np.minimum(np.exp(rng.random(n) * np.log(v + 1)).astype(np.int64), v) - 1
    if kind == "some":
        t[rng.random(n) < 0.3] = -1 - rng.integers(0, 5)
    return t.astype(np.int32)


def _data(n, c, dtype, rng, stride=None):
    buf = torch.from_numpy(rng.standard_normal((n, stride or c)).astype(np.float32)).to(DT[dtype]).cuda()
    return buf[:, :c]


def _ws(desc):
    return torch.full((max(256, stp.stp_embed_workspace_size(desc)),), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,v,c,scale,pad", [(1, 1, 8, 1.0, 0), (7, 5, 8, -0.5, 8), (40, 9, 264, 3.0, 0), (129, 300, 1000, 1.0, 24),
                                             (5000, 77, 16, 8.0, 0), (33, 50000, 4096, 64.0, 0), (3, 4, 65536, 1.0, 0)])
def test_fwd(n, v, c, scale, pad, dtype):
    rng = np.random.default_rng(n + c)
    table = _data(v, c, dtype, rng)
    tok = _tokens("some", n, v, rng)
    desc = stp.embed_desc(n, v, c, dtype, scale, c + pad)
    buf = torch.full((n, c + pad), NAN, dtype=DT[dtype], device="cuda")
    ws = _ws(desc)
    stp.stp_embed_fwd(desc, table, torch.from_numpy(tok).cuda(), buf, ws)
    torch.cuda.synchronize()
    assert stp.stp_device_status(ws) == stp.STP_OK
    want, u = OE.fwd(table.double().cpu().numpy(), tok, scale), torch.finfo(DT[dtype]).eps / 2
    got = buf.double().cpu().numpy()
    assert (np.abs(got[:, :c] - want) <= (2.0 ** -24 + u) * (1 + u) * np.abs(want)).all()
    assert np.isnan(got[:, c:]).all()                   # what lies between is not touched


def _bwd(n, v, c, dtype, tok, scale=1.0, pad=0, add=False, seed=0, stream=None):
    rng = np.random.default_rng(seed + n + c)
    d = _data(n, c, dtype, rng, c + pad) if n else None
    desc = stp.embed_desc(n, v, c, dtype, scale, c + pad)
    start = torch.from_numpy(rng.standard_normal((v, c)).astype(np.float32)).cuda()
    grad = start.clone() if add else torch.full((v, c), NAN, device="cuda")
    ws, t = _ws(desc), torch.from_numpy(tok).cuda()
    if n:
        d.masked_fill_((t < 0)[:, None], NAN)           # not read
    torch.cuda.synchronize()
    stp.stp_embed_bwd(desc, d, t, add, grad, ws, stream=stream)
    torch.cuda.synchronize()
    status = stp.stp_device_status(ws)
    dh = d.double().cpu().numpy() if n else np.zeros((0, c))
    want, size, count = OE.bwd(np.where((tok < 0)[:, None], 0, dh), tok, v, scale)
    tol = (count[:, None] + 2) * 2.0 ** -24 * size
    got = grad.double().cpu().numpy()
    if add:
        want = want + start.double().cpu().numpy()
        assert torch.equal(grad[torch.from_numpy(count == 0).cuda()], start[torch.from_numpy(count == 0).cuda()])
    tol = tol + 2.0 ** -24 * np.abs(want)
    assert (np.abs(got - want) <= tol).all()
    return grad, status


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("kind", ["one", "few", "runs", "zipf", "some"])
@pytest.mark.parametrize("n,v,c", [(1, 1, 8), (31, 40, 16), (32, 2, 8), (33, 600, 264), (1000, 513, 40), (9000, 3000, 520)])
def test_bwd(n, v, c, kind, dtype, add):
    tok = _tokens(kind, n, v, np.random.default_rng(n))
    _, status = _bwd(n, v, c, dtype, tok, 0.75, 8 if c == 40 else 0, add)
    assert status == stp.STP_OK


@pytest.mark.parametrize("v", [1, 2, 255, 256, 257, 511, 512, 513, 65535, 262143, 262144, 300000, 1 << 24])
def test_bwd_vocabularies(v):
    # one, two and three passes of the sort; the last tokens occur
    tok = np.random.default_rng(v).integers(0, v, 3000).astype(np.int32)
    tok[:7] = v - 1
    tok[9] = 0
    assert _bwd(3000, v, 8, stp.STP_BF16, tok)[1] == stp.STP_OK


@pytest.mark.parametrize("n,c", [(70001, 8), (20000, 2056), (300, 16384)])
def test_bwd_large(n, c):
    v = 2000
    tok = _tokens("some", n, v, np.random.default_rng(n))
    assert _bwd(n, v, c, stp.STP_BF16, tok, c ** 0.5)[1] == stp.STP_OK


def test_bwd_is_the_same_each_time_and_on_another_stream():
    tok = _tokens("zipf", 20000, 500, np.random.default_rng(1))
    a, _ = _bwd(20000, 500, 256, stp.STP_FP32, tok)
    b, _ = _bwd(20000, 500, 256, stp.STP_FP32, tok, stream=torch.cuda.Stream())
    assert torch.equal(a, b)


def test_no_token():
    grad, status = _bwd(0, 37, 16, stp.STP_BF16, np.zeros(0, np.int32))
    assert status == stp.STP_OK and not grad.any()
    grad, status = _bwd(50, 37, 16, stp.STP_BF16, np.full(50, -1, np.int32))
    assert status == stp.STP_OK and not grad.any()
    _bwd(50, 37, 16, stp.STP_BF16, np.full(50, -1, np.int32), add=True)
    desc = stp.embed_desc(0, 37, 16)
    ws = _ws(desc)
    stp.stp_embed_fwd(desc, None, None, None, ws)
    assert stp.stp_device_status(ws) == stp.STP_OK


@pytest.mark.parametrize("n", [40, 5000])
def test_a_token_past_the_vocabulary(n):
    rng = np.random.default_rng(n)
    tok = _tokens("zipf", n, 30, rng)
    tok[n // 2] = 30
    tok[n - 1] = 2 ** 31 - 1
    desc = stp.embed_desc(n, 30, 16)
    table, out, ws, t = _data(30, 16, stp.STP_BF16, rng), torch.full((n, 16), NAN, dtype=torch.bfloat16, device="cuda"), _ws(desc), torch.from_numpy(tok).cuda()
    stp.stp_embed_fwd(desc, table, t, out, ws)
    assert stp.stp_device_status(ws) == stp.STP_EDEVICE
    assert not out[n - 1].any() and not out[n // 2].any() and torch.equal(out[0], table[tok[0]])
    _, status = _bwd(n, 30, 16, stp.STP_BF16, tok)      # counts as negative
    assert status == stp.STP_EDEVICE
    stp.stp_embed_fwd(desc, table, t.clamp(max=29), out, ws)
    assert stp.stp_device_status(ws) == stp.STP_OK      # the word is cleared


def test_captured():
    n, v, c = 3000, 700, 264
    rng = np.random.default_rng(0)
    tok = torch.from_numpy(_tokens("some", n, v, rng)).cuda()
    d, desc = _data(n, c, stp.STP_BF16, rng), stp.embed_desc(n, v, c)
    table, out = _data(v, c, stp.STP_BF16, rng), torch.empty(n, c, dtype=torch.bfloat16, device="cuda")
    want_out, want = torch.empty_like(out), torch.empty(v, c, device="cuda")
    ws, grad = _ws(desc), torch.full((v, c), NAN, device="cuda")
    stp.stp_embed_fwd(desc, table, tok, want_out, ws)
    stp.stp_embed_bwd(desc, d, tok, False, want, ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        stp.stp_embed_fwd(desc, table, tok, out, ws)
        stp.stp_embed_bwd(desc, d, tok, False, grad, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want_out) and torch.equal(grad, want)
    # other tokens in the captured buffers
    tok.copy_(torch.from_numpy(_tokens("zipf", n, v, rng)))
    graph.replay()
    stp.stp_embed_bwd(desc, d, tok, False, want, ws)
    torch.cuda.synchronize()
    assert torch.equal(grad, want)
