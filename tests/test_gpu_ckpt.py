"""Activations in 8 bits and the weight gradient from them on the GPU
(stp_ckpt_*) against the float64 oracle (oracle/ckpt.py).

What is kept is defined to the bit, so it is compared for equality.  The
weight gradient's products are exact; its sums of N float32 terms, in any
order, are off by at most N 2^-22 of the sum of magnitudes, and inputs of small whole
numbers, whose sums stay below 2^24, must come out exactly.
"""
import numpy as np
import pytest
import torch

from oracle import ckpt as OC
from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
DT = {stp.STP_BF16: torch.bfloat16, stp.STP_FP32: torch.float32}
NAN, INF = float("nan"), float("inf")


def _space(size):
    return torch.full((max(256, size),), 255, dtype=torch.uint8, device="cuda")


def _strided(x, stride, offset):
    """x on the GPU in a buffer of NaN: rows `stride` apart, `offset` elements in; (view, buffer)."""
    n, c = x.shape
    buf = torch.full((n * stride + offset,), NAN, dtype=x.dtype, device="cuda")
    view = buf[offset:].as_strided((n, c), (stride, 1), offset)
    view.copy_(x)
    return view, buf


def _round_trip(x, stride=None, offset=0, stream=None):
    n, c = x.shape
    stride = c if stride is None else stride
    dtype = stp.STP_BF16 if x.dtype == torch.bfloat16 else stp.STP_FP32
    desc = stp.ckpt_desc(n, c, dtype, stride)
    view, _ = _strided(x, stride, offset)
    out, buf = _strided(torch.zeros_like(x), stride, offset)
    ckpt = _space(stp.stp_ckpt_size(desc))
    torch.cuda.synchronize()
    stp.stp_ckpt_save(desc, view, ckpt, stream=stream)
    stp.stp_ckpt_load(desc, ckpt, out, stream=stream)
    torch.cuda.synchronize()
    between = buf[offset:].as_strided((n - 1, stride - c), (stride, 1), offset + c) if n > 1 and stride > c else buf[:offset]
    assert torch.isnan(between).all() and torch.isnan(buf[:offset]).all()
    return out, ckpt


def _values(n, c, dtype, seed=0):
    rng = np.random.default_rng(seed + n + 7 * c)
    x = rng.standard_normal((n, c)) * np.exp(2 * rng.standard_normal((1, c))) * np.exp(rng.standard_normal((n, 1)))
    x[rng.random((n, c)) < 0.05] = 0
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,c,pad,offset", [(1, 1, 0, 0), (1, 64, 0, 0), (15, 31, 0, 0), (16, 32, 2, 0), (17, 33, 0, 0), (64, 96, 0, 0),
                                            (65, 200, 3, 1), (63, 65, 1, 0), (130, 1000, 0, 0), (3, 5000, 0, 2), (1025, 520, 8, 8),
                                            (2, 65536, 0, 0)])
def test_what_is_kept(n, c, pad, offset, dtype):
    x = _values(n, c, dtype)
    got, _ = _round_trip(x, c + pad, offset)
    assert np.array_equal(got.double().cpu().numpy(), OC.keep(x.double().numpy()))


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
def test_every_bf16_value_and_the_borders_of_scales(dtype):
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    every = every[torch.isfinite(every.float())]
    # alone in a block (its own scale), and beside larger ones (subnormal codes and 0)
    for step in (32, 1):
        k = every.numel() // 64 * 64
        x = torch.zeros(k // 64, 64 * step) if step > 1 else every[:k].float().view(-1, 64)
        if step > 1:
            x[:, ::step] = every[:k].float().view(-1, 64)
        x = x.to(DT[dtype])
        got, _ = _round_trip(x)
        assert np.array_equal(got.double().cpu().numpy(), OC.keep(x.double().numpy()))
    if dtype == stp.STP_FP32:
        top = np.array([448.0, np.nextafter(np.float32(448), np.float32(449)), 1e-38, 1e-40, 3.4e38, 2.0 ** -108, 2.0 ** -117], np.float32)
        x = torch.zeros(7, 32)
        x[:, 5] = torch.from_numpy(top)
        x[:, 9] = torch.from_numpy(-top / 3)
        x[:, 31] = torch.from_numpy(top / 500)
        got, _ = _round_trip(x)
        assert np.array_equal(got.double().cpu().numpy(), OC.keep(x.double().numpy()))


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
def test_infinities_and_nan_keep_to_their_block(dtype):
    x = _values(70, 100, dtype)
    x[3, 40], x[16, 0], x[69, 99] = INF, NAN, -INF
    got, _ = _round_trip(x)
    want = OC.keep(x.double().numpy())
    assert np.isnan(want).sum() == 32 + 32 + 4
    assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)


def test_restored_values_are_kept_unchanged():
    x = _values(100, 300, stp.STP_BF16)
    once, _ = _round_trip(x)
    twice, _ = _round_trip(once.cpu())
    assert torch.equal(once, twice)


# ------------------------------------------------------------ weight gradient

def _wgrad(x, dy, pad=0, add=None, stream=None, times=1):
    n, c = x.shape
    m = dy.shape[1]
    desc = stp.ckpt_desc(n, c, stp.STP_BF16 if x.dtype == torch.bfloat16 else stp.STP_FP32)
    ckpt, ws = _space(stp.stp_ckpt_size(desc)), _space(stp.stp_ckpt_wgrad_workspace_size(desc, m))
    stride = (m + 7) // 8 * 8 + pad
    y = torch.full((n, stride), NAN, dtype=torch.bfloat16, device="cuda")
    y[:, :m] = dy.cuda()
    dw = torch.full((c, m), NAN, device="cuda") if add is None else add.cuda().clone()
    xd = x.cuda()
    torch.cuda.synchronize()
    if n:
        stp.stp_ckpt_save(desc, xd, ckpt, stream=stream)
    for _ in range(times):
        stp.stp_ckpt_wgrad(desc, m, ckpt, y if n else None, stride, add is not None, dw, ws, stream=stream)
    torch.cuda.synchronize()
    assert stp.stp_device_status(ws) == stp.STP_OK
    return dw


def _whole(n, c, m, seed=0):
    rng = np.random.default_rng(seed + n + c + m)
    return (torch.from_numpy(rng.integers(-8, 9, (n, c)).astype(np.float32)).bfloat16(),
            torch.from_numpy(rng.integers(-4, 5, (n, m)).astype(np.float32)).bfloat16())


SIZES = [(1, 1, 1), (1, 128, 256), (64, 32, 16), (63, 33, 17), (65, 127, 255), (64, 129, 257), (200, 300, 523), (512, 256, 1024),
         (1000, 40, 9), (5000, 1000, 100), (129, 2000, 1500), (20001, 130, 300), (70000, 64, 64), (4096, 1300, 5000), (300, 5000, 4100)]


@pytest.mark.parametrize("n,c,m", SIZES)
def test_whole_numbers_exactly(n, c, m):
    x, dy = _whole(n, c, m)
    want = (x.double().T @ dy.double()) if n * c * m < 1e9 else (x.cuda().double().T @ dy.cuda().double()).cpu()
    assert float(want.abs().max()) < 2 ** 24 and 32 * n < 2 ** 24
    assert torch.equal(_wgrad(x, dy).double().cpu(), want)


@pytest.mark.parametrize("n,c,m", [(64, 32, 16), (65, 127, 255), (200, 300, 523), (20001, 130, 300)])
def test_real_values(n, c, m):
    x = _values(n, c, stp.STP_FP32)
    dy = torch.from_numpy(np.random.default_rng(n).standard_normal((n, m)).astype(np.float32)).bfloat16()
    k, d = torch.from_numpy(OC.keep(x.double().numpy())), dy.double()
    got = _wgrad(x, dy).double().cpu()
    assert ((got - k.T @ d).abs() <= n * 2.0 ** -22 * (k.abs().T @ d.abs())).all()


@pytest.mark.parametrize("n,c,m", [(65, 127, 255), (20001, 130, 300), (4096, 1300, 5000), (129, 2000, 1500)])
def test_accumulates(n, c, m):
    x, dy = _whole(n, c, m)
    start = torch.arange(c * m, dtype=torch.float32).remainder(1000).view(c, m)
    want = start.double().cuda() + 2 * (x.cuda().double().T @ dy.cuda().double())
    assert torch.equal(_wgrad(x, dy, pad=8, add=start, times=2).double(), want)


def test_no_token():
    x, dy = torch.zeros(0, 50).bfloat16(), torch.zeros(0, 20).bfloat16()
    assert not _wgrad(x, dy).any()
    start = torch.randn(50, 20)
    assert torch.equal(_wgrad(x, dy, add=start).cpu(), start)


def test_nan_stays_in_its_channels():
    x, dy = _whole(100, 200, 30)
    clean = _wgrad(x, dy)
    x[70, 65] = INF
    got = _wgrad(x, dy)
    assert torch.isnan(got[64:96]).all() and torch.equal(got[:64], clean[:64]) and torch.equal(got[96:], clean[96:])
    x, dy = _whole(100, 200, 30)
    dy[3, 7] = NAN
    got = _wgrad(x, dy)
    assert torch.isnan(got[:, 7]).all() and not torch.isnan(got[:, :7]).any() and not torch.isnan(got[:, 8:]).any()


def test_same_each_time_captured_and_on_another_stream():
    n, c, m = 10001, 500, 700
    x = _values(n, c, stp.STP_BF16)
    dy = torch.randn(n, m, generator=torch.Generator().manual_seed(0)).bfloat16()
    want = _wgrad(x, dy)
    assert torch.equal(_wgrad(x, dy, pad=16, stream=torch.cuda.Stream()), want)
    desc = stp.ckpt_desc(n, c)
    ckpt, ws = _space(stp.stp_ckpt_size(desc)), _space(stp.stp_ckpt_wgrad_workspace_size(desc, m))
    y, xd, dw = torch.empty(n, 704, dtype=torch.bfloat16, device="cuda"), x.cuda(), torch.empty(c, m, device="cuda")
    y[:, :m] = dy.cuda()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        stp.stp_ckpt_save(desc, xd, ckpt)
        stp.stp_ckpt_wgrad(desc, m, ckpt, y, 704, False, dw, ws)
    for _ in range(3):
        dw.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, want)
    assert stp.stp_device_status(ws) == stp.STP_OK


def test_calls_one_behind_another():
    # sizes with and without parts, one after another without waiting, in one workspace
    sizes = [(512, 256, 1024), (20001, 130, 300), (65, 127, 255), (4096, 1300, 5000)]
    data = [_whole(*z) for z in sizes]
    descs = [stp.ckpt_desc(n, c) for n, c, _ in sizes]
    ws = _space(max(stp.stp_ckpt_wgrad_workspace_size(d, z[2]) for d, z in zip(descs, sizes)))
    kept, ys, dws = [], [], []
    for (x, dy), d, (n, c, m) in zip(data, descs, sizes):
        ck = _space(stp.stp_ckpt_size(d))
        stp.stp_ckpt_save(d, x.cuda(), ck)
        y = torch.zeros(n, (m + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda")
        y[:, :m] = dy.cuda()
        kept.append(ck), ys.append(y), dws.append(torch.zeros(c, m, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(5):
        for d, (n, c, m), ck, y, dw in zip(descs, sizes, kept, ys, dws):
            stp.stp_ckpt_wgrad(d, m, ck, y, y.stride(0), True, dw, ws)
    torch.cuda.synchronize()
    assert stp.stp_device_status(ws) == stp.STP_OK
    for (x, dy), dw in zip(data, dws):
        assert torch.equal(dw.double(), 5 * (x.cuda().double().T @ dy.cuda().double()))
