"""Token statistics and distillation on the GPU (stp_token_stats_*,
stp_distill_*) against the float64 oracle (oracle/token_loss.py).

Tolerance.  ln sum exp: 2^x is within 2^-22, its argument within 2^-23 of the
largest |z| log2 e, and the sum of V terms is taken in float32 in chains of at
most V / 256 + 48: e = (V / 256 + 48) 2^-24 + 2^-21 + |z|max 2^-22, on lse and
on each log-probability.  Entropy sums p ln p with the same weights:
e (1 + range), range the largest |ln p| that still has weight (< 40).  A
gradient's p carries e relative; the result is then rounded once (u).  Losses
are q-weighted sums of K <= 256 differences: 2 e + (K + 8) 2^-24 (1 + range).
Ids are exact.
"""
import numpy as np
import pytest
import torch

from oracle import token_loss as OT
from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
DT = {stp.STP_BF16: torch.bfloat16, stp.STP_FP32: torch.float32}
NAN, INF = float("nan"), float("inf")


def _err(z, scale):
    z = np.abs(z[np.isfinite(z)]) * scale
    return lambda v: (v / 256 + 48) * 2.0 ** -24 + 2.0 ** -21 + (z.max() if z.size else 0) * 2.0 ** -22


def _logits(n, v, dtype, seed, offset=0, stride=None, std=3.0):
    """[n, v] view of a buffer: rows `stride` apart, the first `offset` elements in."""
    g = torch.Generator().manual_seed(seed)
    stride = v if stride is None else stride
    buf = (torch.randn(n * stride + offset, generator=g) * std).to(DT[dtype]).cuda()
    return buf[offset:].as_strided((n, v), (stride, 1), offset)


def _stats(z, targets, k, dtype, scale, stride=None, stream=None):
    n, v = z.shape
    d = stp.stats_desc(n, v, k, dtype, scale, stride)
    row = lambda: torch.full((n,), NAN, device="cuda")  # noqa: E731
    out = [row(), row(), row(), torch.full((n, max(k, 1)), -7, dtype=torch.int32, device="cuda"),
           torch.full((n, max(k, 1)), NAN, device="cuda")]
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    t = torch.as_tensor(targets, dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    stp.stp_token_stats_fwd(d, z, t, *out, ws, stream=stream)
    torch.cuda.synchronize()
    return d, t, out, stp.stp_device_status(ws)


def _check_stats(z, targets, k, dtype, scale=1.0, stride=None, stream=None):
    d, t, out, status = _stats(z, targets, k, dtype, scale, stride, stream)
    assert status == stp.STP_OK
    zh = z.double().cpu().numpy()
    e = _err(zh, scale)(z.shape[1])
    lp, ent, lse, ids, top = (x.double().cpu().numpy() for x in out)
    for n in range(len(zh)):
        if targets[n] < 0:
            assert lp[n] == ent[n] == lse[n] == 0
            if k:
                assert (ids[n] == -1).all() and (top[n] == -INF).all()
            continue
        w = OT.stats_row(zh[n], targets[n], k, scale)
        for got, want, tol in ((lp[n], w[0], e), (lse[n], w[2], e), (ent[n], w[1], 41 * e)):
            assert got == want or abs(got - want) <= tol, (n, got, want, tol)
        if k:
            assert ids[n].tolist() == w[3].tolist()
            assert np.array_equal(np.isinf(top[n]), np.isinf(w[4]))
            live = np.isfinite(w[4])
            assert (np.abs(top[n][live] - w[4][live]) <= e).all()
    return d, t, out


def _check_stats_grad(z, targets, d, t, out, dtype, scale, entropy=True, in_place=False, into=None):
    n, v = z.shape
    zh, u = z.double().cpu().numpy(), torch.finfo(DT[dtype]).eps / 2
    rng = np.random.default_rng(0)
    g = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    h = torch.from_numpy(0.1 * rng.standard_normal(n).astype(np.float32)).cuda() if entropy else None
    dz = z if in_place else into if into is not None else torch.full_like(z, NAN)
    lse, ent = out[2].clone(), out[1].clone()
    stp.stp_token_stats_bwd(d, z, t, lse, ent, g, h, dz)
    torch.cuda.synchronize()
    got, e = dz.double().cpu().numpy(), _err(zh, scale)(v)
    for r in range(n):
        if targets[r] < 0:
            assert (got[r] == 0).all()
            continue
        gr, hr = float(g[r]), float(h[r]) if entropy else 0.0
        want = OT.stats_grad_row(zh[r], targets[r], gr, hr, scale)
        p = np.exp(OT._log_softmax(zh[r] * scale)[0])
        tol = u * np.abs(want) + scale * p * (abs(gr) + 82 * abs(hr)) * 2 * e + 2.0 ** -22 * scale * abs(gr) + 1e-30
        assert (np.abs(got[r] - want) <= tol).all(), r


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,v,k,scale", [
    (1, 1, 1, 1.0), (3, 5, 5, 1.0), (2, 7, 9, 0.5), (4, 8, 1, 1.0), (2, 9, 32, 2.0), (5, 257, 3, 1.0), (33, 1000, 0, 1.0),
    (2, 2048, 32, 1.0), (1, 2049, 8, 1.3), (1, 32003, 20, 1.0),       # odd: rows start anywhere
    (3, 151936, 32, 1.0),                                             # eight blocks to a row
    (9, 8193, 5, 1.0), (700, 640, 2, 1.0), (700, 641, 32, 0.7),       # one block to a row
])
def test_stats_match_oracle(n, v, k, scale, dtype):
    z = _logits(n, v, dtype, seed=n + v + k)
    targets = np.random.default_rng(v).integers(0, v, n)
    if n > 2:
        targets[1] = -1
        z[1] = NAN                                                    # not read
    d, t, out = _check_stats(z, targets, k, dtype, scale)
    _check_stats_grad(z, targets, d, t, out, dtype, scale)


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("offset,stride", [(1, 1001), (3, 1007), (5, 1024), (0, 2000)])
def test_strided_rows_of_any_alignment(offset, stride, dtype):
    z = _logits(6, 1001, dtype, seed=offset, offset=offset, stride=stride)
    targets = [0, 1000, 5, 500, 999, 1]
    d, t, out = _check_stats(z, targets, 7, dtype, 1.0, stride)
    other = torch.full((6 * stride + 8,), NAN, dtype=DT[dtype], device="cuda")
    for shift in (offset, offset + 1, offset + 2):                    # the gradient's rows aligned alike, and not
        into = other[shift:].as_strided((6, 1001), (stride, 1), shift)
        _check_stats_grad(z, targets, d, t, out, dtype, 1.0, into=into)
        used = torch.zeros_like(other, dtype=torch.bool)
        used.as_strided((6, 1001), (stride, 1), shift).fill_(True)
        assert torch.isnan(other[~used]).all()                        # nothing between the rows is touched
        other.fill_(NAN)
    _check_stats_grad(z, targets, d, t, out, dtype, 1.0, in_place=True)


@pytest.mark.parametrize("n", [2, 640])
def test_masked_tied_and_empty_rows(n):
    v = 5000
    z = _logits(n, v, stp.STP_BF16, seed=1)
    targets = np.arange(n) * 7 % v
    z[:, 3000:] = -INF                     # a padded vocabulary
    z[0] = 1.5                             # all equal: the smallest ids
    targets[0] = v - 1
    z[1] = -INF                            # nothing left
    if n > 2:
        z[2] = -INF
        z[2, 4321] = -80.0                 # one token alone
        z[3, :] = torch.tensor([0.0, -0.0] * (v // 2))       # equal too
        z[4] = torch.arange(v, device="cuda").to(torch.bfloat16)             # ascending, with ties
        z[5] = -torch.arange(v, device="cuda").to(torch.bfloat16)
        z[6, 8:16] = 30.0                  # the largest all in one piece of the row
        z[7, ::2048] = 29.0                # the largest all in one thread's strip
        z[8] = 3e38                        # at the type's ends
        z[9] = -3e38
        targets[2], targets[8], targets[9] = 4321, 3, 4
    d, t, out = _check_stats(z, targets, 32, stp.STP_BF16)
    ok = torch.tensor([r != 1 for r in range(n)])
    _check_stats_grad(z[ok.cuda()].contiguous(), targets[ok.numpy()],
                      stp.stats_desc(n - 1, v, 0), t[ok.cuda()].contiguous(), [x[ok.cuda()].contiguous() for x in out],
                      stp.STP_BF16, 1.0)


def test_rows_with_nan_or_infinity():
    z = _logits(4, 3000, stp.STP_FP32, seed=2)
    z[0, 17], z[1, 2999], z[2] = NAN, INF, NAN
    _, _, out, status = _stats(z, [5, 6, 7, 8], 3, stp.STP_FP32, 1.0)
    assert status == stp.STP_OK
    for x in (out[0], out[1], out[2]):
        assert torch.isnan(x[:3]).all() and torch.isfinite(x[3])
    assert torch.isnan(out[4][:2]).all() and torch.isfinite(out[4][3]).all()


def test_targets_outside_the_vocabulary():
    z = _logits(3, 1000, stp.STP_BF16, seed=3)
    d, t, out, status = _stats(z, [999, 1000, 2 ** 31 - 1], 1, stp.STP_BF16, 1.0)
    assert status == stp.STP_EDEVICE
    assert torch.isfinite(out[0][0]) and torch.isnan(out[0][1:]).all() and torch.isfinite(out[2]).all()
    dz, g = torch.full_like(z, NAN), torch.ones(3, device="cuda")
    stp.stp_token_stats_bwd(d, z, t, out[2], out[1], g, g, dz)
    torch.cuda.synchronize()
    assert torch.isfinite(dz).all() and (dz[1:] == 0).all()
    assert _stats(z, [1, 2, 3], 1, stp.STP_BF16, 1.0)[3] == stp.STP_OK      # the word is cleared


@pytest.mark.parametrize("n", [1, 30, 640])
def test_stats_same_bits_again_and_on_another_stream(n):
    z = _logits(n, 20011, stp.STP_BF16, seed=n)
    targets = np.arange(n)
    runs = [_stats(z, targets, 9, stp.STP_BF16, 1.0, stream=s)[2] for s in (None, None, torch.cuda.Stream())]
    for a, b, c in zip(*runs):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_no_rows():
    z = torch.empty(0, 10, dtype=torch.bfloat16, device="cuda")
    assert _stats(z, [], 2, stp.STP_BF16, 1.0)[3] == stp.STP_OK


# ------------------------------------------------------------------ distillation

def _teacher(n, v, k, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.choice(v, k, replace=False) if v >= k else rng.integers(0, v, k) for _ in range(n)]).astype(np.int32)
    return ids, (rng.standard_normal((n, k)) * 2).astype(np.float32)


def _distill(z, ids, tl, mask, dtype, scale, how, stride=None, into=None, stream=None):
    n, v = z.shape
    d = stp.distill_desc(n, v, ids.shape[1], dtype, scale, stride)
    i, t = torch.from_numpy(ids).cuda(), torch.from_numpy(tl).cuda()
    m = None if mask is None else torch.from_numpy(mask).cuda()
    g = torch.from_numpy(np.random.default_rng(4).standard_normal(n).astype(np.float32)).cuda()
    loss, lse = torch.full((n,), NAN, device="cuda"), torch.full((n,), NAN, device="cuda")
    dz = torch.full_like(z, NAN) if into is None else into
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    if how == "step":
        stp.stp_distill_step(d, z, i, t, m, g, loss, lse, dz, ws, stream=stream)
    else:
        stp.stp_distill_fwd(d, z, i, t, m, loss, lse, ws, stream=stream)
        stp.stp_distill_bwd(d, z, i, t, m, lse, g, dz, stream=stream)
    torch.cuda.synchronize()
    return g, loss, lse, dz, stp.stp_device_status(ws)


def _check_distill(z, ids, tl, mask, dtype, scale=1.0, how="step", stride=None, into=None):
    zh, u = z.double().cpu().numpy(), torch.finfo(DT[dtype]).eps / 2
    g, loss, lse, dz, status = _distill(z, ids, tl, mask, dtype, scale, how, stride, into)
    assert status == stp.STP_OK
    e, k = _err(zh, scale)(z.shape[1]), ids.shape[1]
    loss, lse, dz = (x.double().cpu().numpy() for x in (loss, lse, dz))
    for n in range(len(zh)):
        on = (mask is None or mask[n]) and ((ids[n] >= 0) & (tl[n] > -INF)).any()
        if not on:
            assert loss[n] == lse[n] == 0 and (dz[n] == 0).all()
            continue
        w, wl = OT.distill_row(zh[n], ids[n], tl[n], scale)
        a = np.abs(tl[n][np.isfinite(tl[n])]).max() * scale
        assert loss[n] == w or abs(loss[n] - w) <= 2 * e + (k + 8) * 2.0 ** -24 * 41 + a * 2.0 ** -21, (n, loss[n], w)
        assert abs(lse[n] - wl) <= e
        want, gn = OT.distill_grad_row(zh[n], ids[n], tl[n], float(g[n]), scale), abs(float(g[n])) * scale
        p = np.exp(OT._log_softmax(zh[n] * scale)[0])
        q = np.zeros(len(p))
        np.add.at(q, ids[n][ids[n] >= 0], OT._teacher(ids[n], tl[n], scale)[1][ids[n] >= 0])
        tol = u * np.abs(want) + gn * (2 * e * p + ((k + 16) * 2.0 ** -24 + a * 2.0 ** -21) * q) + 1e-30
        assert (np.abs(dz[n] - want) <= tol).all(), n


@pytest.mark.parametrize("how", ["step", "two"])
@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,v,k,scale", [(1, 1, 1, 1.0), (2, 5, 3, 1.0), (3, 100, 100, 0.5), (5, 1000, 64, 1.0),
                                         (2, 40001, 256, 2.0), (1, 151936, 64, 1.0), (640, 777, 33, 1.0)])
def test_distill_matches_oracle(n, v, k, scale, dtype, how):
    z = _logits(n, v, dtype, seed=v + k)
    ids, tl = _teacher(n, v, k, seed=n)
    _check_distill(z, ids, tl, None, dtype, scale, how)


@pytest.mark.parametrize("how", ["step", "two"])
def test_absent_repeated_and_masked_entries(how):
    n, v, k = 12, 3001, 40
    z = _logits(n, v, stp.STP_FP32, seed=6)
    ids, tl = _teacher(n, v, k, seed=6)
    mask = np.ones(n, np.uint8)
    ids[0, 5:] = -1
    ids[1] = -1                                # lists nothing
    ids[2] = 17                                # one id, k times
    ids[3, ::2] = ids[3, 1]                    # and half the times
    tl[4, :39] = -INF                          # a single entry is left
    tl[5] = -INF
    ids[6, 0] = -2 ** 31
    mask[7], mask[8] = 0, 255
    z[7] = NAN                                 # not read
    z[9, ids[9][1:]] = -INF                    # the student rules listed ids out
    tl[9, 1:] = -INF                           # ... which the teacher does too
    tl[10] += 1000.0
    _check_distill(z, ids, tl, mask, stp.STP_FP32, 1.0, how)


@pytest.mark.parametrize("how", ["step", "two"])
def test_rows_of_the_types_lowest_value(how):
    """Masks that use the lowest finite value instead of -inf: probability 0 next
    to others, and an even distribution in a row of nothing else."""
    low, n, v, k = torch.finfo(torch.float32).min, 4, 700, 6
    z = _logits(n, v, stp.STP_FP32, seed=3)
    ids, tl = _teacher(n, v, k, seed=3)
    z[0, 10:] = low
    ids[0] = np.arange(k)
    tl[1, 2:] = low
    tl[2] = low
    z[3] = low
    g, loss, lse, dz, status = _distill(z, ids, tl, None, stp.STP_FP32, 1.5, how)
    assert status == stp.STP_OK
    # e of the values that count, |z| < 16 * 1.5: under 1e-5; twice that and K terms of it on the loss
    zh = z.double().cpu().numpy()
    for r in range(3):
        want = OT.distill_row(zh[r], ids[r], tl[r], 1.5)[0]
        assert abs(float(loss[r]) - want) <= 4e-5, r
        off = np.abs(dz[r].double().cpu().numpy() - OT.distill_grad_row(zh[r], ids[r], tl[r], float(g[r]), 1.5))
        assert off.max() <= 4e-5 * abs(float(g[r])) * 1.5, r
    # every token alike: ln V - (entropy of q); the sum of V exponentials is exact here
    q = OT._teacher(ids[3], tl[3], 1.5)[1]
    assert abs(float(loss[3]) - (np.log(v) + (q * np.log(q)).sum())) < 1e-4
    d, t, out, _ = _stats(z, [0, 1, 2, 3], 3, stp.STP_FP32, 1.5)
    assert abs(float(out[0][3]) + np.log(v)) < 1e-5 and abs(float(out[1][3]) - np.log(v)) < 1e-5
    assert out[3][3].tolist() == [0, 1, 2]


@pytest.mark.parametrize("n", [2, 640])
def test_gradients_of_rows_of_nothing(n):
    """Rows of nothing but -inf: no distribution, a gradient of zeros, the others untouched."""
    v = 4000
    z = _logits(n, v, stp.STP_BF16, seed=5)
    z[1] = -INF
    ids, tl = _teacher(n, v, 5, seed=5)
    for how in ("step", "two"):
        _, loss, lse, dz, status = _distill(z, ids, tl, None, stp.STP_BF16, 1.0, how)
        assert status == stp.STP_OK and loss[1] == INF and lse[1] == -INF
        assert (dz[1] == 0).all() and torch.isfinite(dz).all() and (dz[0] != 0).any()
    d, t, out, _ = _stats(z, np.zeros(n, int), 2, stp.STP_BF16, 1.0)
    g, dz = torch.ones(n, device="cuda"), torch.full_like(z, NAN)
    stp.stp_token_stats_bwd(d, z, t, out[2], out[1], g, g, dz)
    torch.cuda.synchronize()
    assert (dz[1] == 0).all() and torch.isfinite(dz).all() and (dz[0] != 0).any()


def test_infinite_loss():
    z = _logits(1, 500, stp.STP_FP32, seed=1)
    z[0, 7] = -INF
    _, loss, lse, dz, _ = _distill(z, np.array([[7, 8]], np.int32), np.zeros((1, 2), np.float32), None, stp.STP_FP32, 1.0, "two")
    assert loss[0] == INF and torch.isfinite(lse).all() and torch.isfinite(dz).all()


def test_ids_outside_the_vocabulary():
    z = _logits(2, 500, stp.STP_BF16, seed=1)
    ids, tl = np.array([[3, 500], [1, 2]], np.int32), np.zeros((2, 2), np.float32)
    for how in ("step", "two"):
        _, loss, _, dz, status = _distill(z, ids, tl, None, stp.STP_BF16, 1.0, how)
        assert status == stp.STP_EDEVICE
        assert abs(float(loss[0]) + OT.stats_row(z[0].double().cpu().numpy(), 3)[0]) < 1e-4     # counts as absent
        assert torch.isfinite(dz).all()
    _, _, _, _, status = _distill(z, ids % 500, tl, None, stp.STP_BF16, 1.0, "step")
    assert status == stp.STP_OK


@pytest.mark.parametrize("how", ["step", "two"])
@pytest.mark.parametrize("n", [3, 640])
def test_distill_strided_in_place_and_misaligned(n, how):
    v, stride = 2003, 2011
    ids, tl = _teacher(n, v, 9, seed=8)
    for dtype in DT:
        z = _logits(n, v, dtype, seed=9, offset=3, stride=stride)
        other = torch.full((n * stride + 8,), NAN, dtype=DT[dtype], device="cuda")
        _check_distill(z, ids, tl, None, dtype, 1.0, how, stride, other[2:].as_strided((n, v), (stride, 1), 2))
        _check_distill(z, ids, tl, None, dtype, 1.0, how, stride, z)


@pytest.mark.parametrize("n", [2, 640])
def test_distill_same_bits_again_and_captured(n):
    z = _logits(n, 12345, stp.STP_BF16, seed=n)
    ids, tl = _teacher(n, 12345, 50, seed=n)
    a, b = (_distill(z, ids, tl, None, stp.STP_BF16, 1.0, "step") for _ in range(2))
    for x, y in zip(a[1:4], b[1:4]):
        assert torch.equal(x, y)
    d = stp.distill_desc(n, 12345, 50)
    i, t, loss, lse, dz = torch.from_numpy(ids).cuda(), torch.from_numpy(tl).cuda(), a[1].clone(), a[2].clone(), torch.empty_like(z)
    ws, g = torch.empty(256, dtype=torch.uint8, device="cuda"), torch.cuda.CUDAGraph()
    loss.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        stp.stp_distill_step(d, z, i, t, None, a[0], loss, lse, dz, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, a[1]) and torch.equal(dz, a[3])


def test_gradients_against_differences():
    z = _logits(2, 300, stp.STP_FP32, seed=4, std=1.0)
    ids, tl = _teacher(2, 300, 5, seed=2)
    g, _, _, dz, _ = _distill(z, ids, tl, None, stp.STP_FP32, 1.0, "two")
    zh = z.double().cpu().numpy()
    for r, c in ((0, int(ids[0, 0])), (1, 0), (1, 299)):
        a, b = zh[r].copy(), zh[r].copy()
        a[c] += 1e-5
        b[c] -= 1e-5
        diff = (OT.distill_row(a, ids[r], tl[r])[0] - OT.distill_row(b, ids[r], tl[r])[0]) / 2e-5 * float(g[r])
        assert abs(float(dz[r, c]) - diff) <= 1e-6 + 1e-4 * abs(diff)
