"""q/k norm with rotation on the GPU (stp_qk_norm_rope_fwd / _bwd) against the
float64 oracle (oracle/qk.py) on the same inputs.

Tolerance: an output is rounded once (half a step, u = eps / 2 of its type)
after float32 work.  Of that, the sum of squares of D <= 512 channels, the
reciprocal root and the three products are each within a few 2^-24 of their
value, the angle within 2^-25 half turns and the sine and cosine within a few
2^-24: W = 64 * 2^-24 of the largest terms covers it.  dw sums N H products
(float32, in chains of under 64 terms joined pairwise): 96 * 2^-24 of the sum
of their absolute values.
"""
import numpy as np
import pytest
import torch

from oracle import qk as OQ
from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
WORK = 64 * 2.0 ** -24


def _case(n, hq, hkv, d, rot, inter, dtype, seed, far=100000):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == stp.STP_BF16 else torch.float32
    width = (hq + 2 * hkv) * d
    c = dict(n=n, hq=hq, hkv=hkv, d=d, rot=rot, inter=inter, dtype=dtype, dt=dt)
    c["qkv"] = torch.randn(n, width, generator=g).to(dt)
    c["dq"], c["dk"] = torch.randn(n, hq, d, generator=g).to(dt), torch.randn(n, hkv, d, generator=g).to(dt)
    c["wq"], c["wk"] = 1 + 0.3 * torch.randn(d, generator=g), 1 + 0.3 * torch.randn(d, generator=g)
    c["pos"] = torch.from_numpy(rng.integers(0, far, n).astype(np.int32))
    c["freq"] = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    c["desc"] = stp.qk_desc(n, hq, hkv, d, rot, inter, dtype, q_stride=width, k_stride=width)
    return c


def _gpu(c, backward=True, stream=None):
    hq, hkv, d, n, dt = c["hq"], c["hkv"], c["d"], c["n"], c["dt"]
    x = c["qkv"].cuda()
    q, k = x[:, :hq * d], x[:, hq * d:]
    pos, wq, wk = (c[y].cuda() if c[y] is not None else None for y in ("pos", "wq", "wk"))
    qo, ko = torch.empty(n, hq, d, dtype=dt, device="cuda"), torch.empty(n, hkv, d, dtype=dt, device="cuda")
    torch.cuda.synchronize()
    stp.stp_qk_norm_rope_fwd(c["desc"], q, k, wq, wk, c["freq"], pos, qo, ko, stream=stream)
    out = {"q": qo, "k": ko}
    if backward:
        dx = torch.full_like(x, 7.0)
        dwq, dwk = torch.full((d,), float("nan"), device="cuda"), torch.full((d,), float("nan"), device="cuda")
        ws = torch.empty(stp.stp_qk_norm_rope_workspace_size(c["desc"]), dtype=torch.uint8, device="cuda")
        dq, dk = c["dq"].cuda(), c["dk"].cuda()
        torch.cuda.synchronize()
        stp.stp_qk_norm_rope_bwd(c["desc"], q, k, wq, wk, c["freq"], pos, dq, dk, dx[:, :hq * d],
                                 dx[:, hq * d:(hq + hkv) * d], dwq, dwk, ws, stream=stream)
        out.update(dx=dx, dwq=dwq, dwk=dwk)
    torch.cuda.synchronize()
    return {y: v.double().cpu().numpy() for y, v in out.items()}


def _check(c, got):
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    u = torch.finfo(c["dt"]).eps / 2
    x = c["qkv"].double().numpy().reshape(n, hq + 2 * hkv, d)
    for name, hs, w, dy in (("q", slice(0, hq), c["wq"], c["dq"]), ("k", slice(hq, hq + hkv), c["wk"], c["dk"])):
        xs, w = x[:, hs], np.ones(d) if w is None else w.double().numpy()
        y = OQ.forward(xs, w, c["pos"], c["freq"], c["rot"], c["inter"])
        big = np.abs(xs * w).max() / np.sqrt((xs ** 2).mean(-1) + 1e-6).min()
        assert (np.abs(got[name] - y) <= u * np.abs(y) + WORK * big).all(), name
        if "dx" in got:
            dy = dy.double().numpy()
            dx, dw = OQ.backward(xs, w, c["pos"], c["freq"], c["rot"], dy, c["inter"])
            mine = got["dx"].reshape(n, hq + 2 * hkv, d)[:, hs]
            r = 1 / np.sqrt((xs ** 2).mean(-1, keepdims=True) + 1e-6)
            big = (np.abs(dy).max(-1, keepdims=True) * 1.5 * np.abs(w).max() * r) * (1 + np.abs(xs * r))
            assert (np.abs(mine - dx) <= u * np.abs(dx) + 4 * WORK * big).all(), "dx " + name
            terms = 1.5 * np.abs(dy).max() * np.abs(xs * r).sum((0, 1))
            assert (np.abs(got["dw" + name] - dw) <= 96 * 2.0 ** -24 * terms).all(), "dw " + name
    if "dx" in got:      # what lies beside the queries and keys stays as it was
        assert (got["dx"].reshape(n, hq + 2 * hkv, d)[:, hq + hkv:] == 7.0).all()


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,hq,hkv,d,rot,inter", [
    (1, 1, 1, 16, 16, False),         # one token, one lane per head
    (1, 32, 8, 128, 128, False),      # a decoding step
    (3, 7, 1, 32, 16, True),
    (5, 3, 2, 48, 48, False),         # three of four lanes work
    (37, 5, 5, 80, 32, False),
    (64, 8, 2, 64, 64, True),
    (129, 9, 3, 96, 0, False),        # no rotation
    (33, 2, 1, 192, 64, True),
    (17, 4, 1, 256, 256, False),
    (9, 2, 2, 512, 512, True),
    (9, 2, 1, 512, 496, False),
    (5000, 4, 1, 64, 64, False),      # every head of a token in one work item
])
def test_matches_oracle(n, hq, hkv, d, rot, inter, dtype):
    c = _case(n, hq, hkv, d, rot, inter, dtype, seed=n + d + rot)
    _check(c, _gpu(c))


def test_packed_row_of_the_benchmark():
    c = _case(1200, 32, 8, 128, 128, False, stp.STP_BF16, seed=5)
    _check(c, _gpu(c))


@pytest.mark.parametrize("n,hq,hkv,d", [(200, 4, 2, 64), (5000, 4, 2, 64)])
def test_same_bits_again_and_on_another_stream(n, hq, hkv, d):
    c = _case(n, hq, hkv, d, d, False, stp.STP_BF16, seed=1)
    a, b, s = _gpu(c), _gpu(c), _gpu(c, stream=torch.cuda.Stream())
    for x in a:
        assert np.array_equal(a[x], b[x]) and np.array_equal(a[x], s[x])


def test_far_positions_and_any_frequency():
    """Positions to 2^31 - 1 and below 0, frequencies above a radian and negative."""
    c = _case(64, 2, 1, 64, 64, False, stp.STP_FP32, seed=3)
    c["pos"][:4] = torch.tensor([2 ** 31 - 1, 0, -5, -(2 ** 31)], dtype=torch.int32)
    c["freq"][:3] = [3.0, -0.5, 50.0]
    # the oracle's own angle, a float64 product, is off by 2^-53 of up to 1.1e11 radians: 1e-5
    got, u = _gpu(c, backward=False), 2.0 ** -24
    x = c["qkv"].double().numpy().reshape(64, 4, 64)
    y = OQ.forward(x[:, :2], c["wq"].double().numpy(), c["pos"], c["freq"], 64)
    assert (np.abs(got["q"] - y) <= u * np.abs(y) + 8 * 1.3e-5).all()


def test_null_weights_zero_vectors_and_in_place():
    c = _case(40, 2, 2, 64, 64, False, stp.STP_FP32, seed=4)
    c["wq"] = c["wk"] = None
    c["qkv"][7] = 0.0                  # the norm of nothing: eps alone
    _check(c, _gpu(c))
    d = stp.qk_desc(40, 2, 2, 64, dtype=stp.STP_FP32)
    q, k = c["qkv"][:, :128].contiguous().cuda(), c["qkv"][:, 128:256].contiguous().cuda()
    pos, qo, ko = c["pos"].cuda(), torch.empty_like(q), torch.empty_like(k)
    stp.stp_qk_norm_rope_fwd(d, q, k, None, None, c["freq"], pos, qo, ko)
    stp.stp_qk_norm_rope_fwd(d, q, k, None, None, c["freq"], pos, q, k)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_no_token_gives_a_zero_weight_gradient():
    d = stp.qk_desc(0, 2, 2, 64)
    dw = torch.full((2, 64), 3.0, device="cuda")
    stp.stp_qk_norm_rope_bwd(d, None, None, None, None, np.ones(32), None, None, None, None, None, dw[0], dw[1], None)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_gradient_against_differences():
    c = _case(3, 2, 1, 32, 32, True, stp.STP_FP32, seed=8, far=50)
    got = _gpu(c)

    def loss(qkv):
        x = qkv.reshape(3, 4, 32)
        return sum((OQ.forward(x[:, h], w.double().numpy(), c["pos"], c["freq"], 32, True) * dy.double().numpy()).sum()
                   for h, w, dy in ((slice(0, 2), c["wq"], c["dq"]), (slice(2, 3), c["wk"], c["dk"])))

    base = c["qkv"].double().numpy()
    for i, j in ((0, 0), (1, 40), (2, 95), (0, 66)):
        a, b = base.copy(), base.copy()
        a[i, j] += 1e-5
        b[i, j] -= 1e-5
        diff = (loss(a) - loss(b)) / 2e-5
        assert abs(got["dx"][i, j] - diff) <= 2e-5 * max(1.0, abs(diff))
