"""Clipped policy loss on the GPU (stp_policy_*) against the float64 oracle
(oracle/policy.py).

Tolerance.  e, the error of a log-probability and of lse, is that of the token
statistics: (V / 256 + 48) 2^-24 + 2^-21 + |z|max 2^-22; the entropy's is 41 e.
The ratio's exponent is a difference of float32 values, so r is off by
r (e + |lp| 2^-23 + 2^-22); likewise exp(ref - lp).  The loss adds three such
terms (2^-22 of their sizes).  A gradient is p (h ln p + c) + g [target]: p
carries 2 e relative, |ln p| < 40 where p counts, c and g the errors above, and
one rounding u.
"""
import numpy as np
import pytest
import torch

from oracle import policy as OP
from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
DT = {stp.STP_BF16: torch.bfloat16, stp.STP_FP32: torch.float32}
NAN, INF = float("nan"), float("inf")
NAMES = ("loss", "logprob", "entropy", "lse", "kl")


class Case:
    def __init__(self, n, v, dtype, scale=1.0, kl=0.3, ent=0.1, low=0.2, high=0.28, seed=0, stride=None, offset=0, z=None):
        rng = np.random.default_rng(seed + 1000 * n + v)
        stride = v if stride is None else stride
        self.n, self.v, self.dtype, self.scale, self.kl, self.ent, self.low, self.high = n, v, dtype, scale, kl, ent, low, high
        buf = torch.from_numpy(rng.standard_normal(n * stride + offset).astype(np.float32) * 3).to(DT[dtype]).cuda()
        self.z = buf[offset:].as_strided((n, v), (stride, 1), offset)
        if z is not None:
            self.z.copy_(z)
        self.zh = self.z.double().cpu().numpy().copy()
        self.t = rng.integers(0, v, n).astype(np.int32)
        if n > 2:
            self.t[1] = -1
        lp = np.array([OP.row(self.zh[i], max(0, self.t[i]), 0.0, None, 0.0, low, high, 0.0, 0.0, scale)[1] for i in range(n)])
        lp = np.where(np.isfinite(lp), lp, -3.0)
        move = rng.standard_normal(n) * 0.3
        for edge in (np.log(1 - low) if low < 1 else -1e9, np.log(1 + high)):
            move = np.where(np.abs(move - edge) < 1e-2, move + 3e-2, move)     # the gradient jumps at a border
        self.old = (lp - move).astype(np.float32)
        self.ref = (lp + rng.standard_normal(n) * 0.4).astype(np.float32) if kl is not None else None
        self.adv = rng.standard_normal(n).astype(np.float32)
        if n > 3:
            self.adv[2] = 0
        self.w = rng.uniform(0.5, 1.5, n).astype(np.float32)
        self.desc = stp.policy_desc(n, v, dtype, scale, low, high, kl or 0.0, ent, stride)

    def want(self, i):
        return OP.row(self.zh[i], self.t[i], float(self.old[i]), None if self.ref is None else float(self.ref[i]), float(self.adv[i]),
                      float(np.float32(self.low)), float(np.float32(self.high)), float(np.float32(self.kl or 0)), float(np.float32(self.ent)),
                      float(np.float32(self.scale)))

    def given(self):
        dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
        return self.z, dev(self.t), dev(self.old), dev(self.ref), dev(self.adv)

    def call(self, how, into=None, stream=None):
        out = {k: torch.full((self.n,), NAN, device="cuda") for k in NAMES}
        ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
        given, w = self.given(), torch.from_numpy(self.w).cuda()
        stride = self.z.stride(0)
        dz = into if into is not None else torch.full((self.n * stride,), NAN, dtype=self.z.dtype, device="cuda").view(self.n, stride)[:, :self.v]
        torch.cuda.synchronize()
        if how == "step":
            stp.stp_policy_step(self.desc, *given, w, *out.values(), dz, ws, stream=stream)
        else:
            stp.stp_policy_fwd(self.desc, *given, *out.values(), ws, stream=stream)
            if how == "both":
                stp.stp_policy_bwd(self.desc, *given, out["logprob"], out["entropy"], out["lse"], w, dz, stream=stream)
        torch.cuda.synchronize()
        self.status = stp.stp_device_status(ws)
        out = {k: x.double().cpu().numpy() for k, x in out.items()}
        if how != "fwd":
            out["dz"] = dz.double().cpu().numpy()
        return out

    def check(self, got, status=stp.STP_OK):
        assert self.status == status
        u, live = torch.finfo(DT[self.dtype]).eps / 2, np.abs(self.zh[np.isfinite(self.zh)]) * self.scale
        e = (self.v / 256 + 48) * 2.0 ** -24 + 2.0 ** -21 + (live.max() if live.size else 0) * 2.0 ** -22
        for i in range(self.n):
            if self.t[i] < 0:
                assert all((x[i] == 0).all() for x in got.values()), i
                continue
            loss, lp, ent, lse, kl, dz = self.want(i)
            a, x = abs(float(self.adv[i])), 0.0 if self.ref is None else float(self.ref[i]) - lp
            f = e + abs(lp) * 2.0 ** -23 + 2.0 ** -22
            b = self.kl or 0.0
            near = {"logprob": (lp, e), "lse": (lse, e), "entropy": (ent, 41 * e),
                    "kl": (kl, abs(np.expm1(x)) * f + 2.0 ** -22 * kl + 1e-30)}
            r = np.exp(lp - self.old[i])
            near["loss"] = (loss, a * min(r, 1 + self.high) * f + b * near["kl"][1] + abs(self.ent) * 41 * e +
                            2.0 ** -22 * (a * min(r, 1 + self.high) + a + b * kl + abs(self.ent * ent)))
            for k, (want, tol) in near.items():
                assert got[k][i] == want or abs(got[k][i] - want) <= tol, (k, i, got[k][i], want, tol)
            if "dz" in got:
                g = OP.terms(lp, ent, float(self.old[i]), None if self.ref is None else float(self.ref[i]), float(self.adv[i]),
                             self.low, self.high, b, self.ent)[2]
                dg = (a * r + b * np.exp(x)) * f + 2.0 ** -22 * (a * r + b * (1 + np.exp(x)))
                p = np.exp(self.zh[i] * self.scale - lse)
                hot = np.arange(self.v) == self.t[i]
                w = float(self.w[i])
                want = w * dz
                tol = u * np.abs(want) + w * self.scale * (p * (abs(g) + 82 * abs(self.ent)) * 2 * e + (p + hot) * (dg + 2.0 ** -22 * abs(g))
                                                            + p * abs(self.ent) * 41 * e) + 1e-30
                assert (np.abs(got["dz"][i] - want) <= tol).all(), (i, np.abs(got["dz"][i] - want).max())


@pytest.mark.parametrize("how", ["fwd", "both", "step"])
@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,v,scale,kl,ent", [
    (1, 1, 1.0, 0.3, 0.1), (3, 5, 1.0, None, 0.0), (5, 257, 0.7, 0.3, -0.2), (33, 1000, 1.0, 0.0, 0.1),
    (1, 32003, 1.0, 0.3, 0.0),                                        # odd: rows start anywhere
    (3, 151936, 1.25, 0.1, 0.01),                                     # eight blocks to a row
    (700, 641, 1.0, 0.3, 0.1),                                        # one block to a row
    (5000, 9, 1.0, 0.3, 0.1),                                         # every row checks its own target
])
def test_matches_oracle(n, v, scale, kl, ent, dtype, how):
    c = Case(n, v, dtype, scale, kl, ent)
    if n > 2:
        c.z[1] = NAN                                                  # not read
    c.check(c.call(how))


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("how", ["both", "step"])
def test_strided_rows_in_place_and_elsewhere(dtype, how):
    for v in (33, 40000):                                             # one and several blocks to a row
        c = Case(6, v, dtype, stride=v + 5, offset=3)
        keep = c.z.clone()
        between = c.z.as_strided((5, 5), (v + 5, 1), c.z.storage_offset() + v).clone()
        a = c.call(how)
        assert torch.equal(c.z, keep)
        c.check(a)
        b = c.call(how, into=c.z)
        assert all(np.array_equal(a[k], b[k]) for k in a)
        assert torch.equal(c.z.as_strided((5, 5), (v + 5, 1), c.z.storage_offset() + v), between)
        other = torch.full((6 * (v + 5) + 1,), NAN, dtype=DT[dtype], device="cuda")[1:].as_strided((6, v), (v + 5, 1), 1)
        c.z.copy_(keep)
        assert np.array_equal(c.call(how, into=other)["dz"], a["dz"])


@pytest.mark.parametrize("how", ["both", "step"])
def test_border_belongs_to_the_unclipped_side(how):
    c = Case(8, 500, stp.STP_FP32, kl=None, ent=0.0, low=0.0, high=0.0)
    c.adv = np.array([1, 1, -1, -1, 2, 2, -2, 0], np.float32)
    c.t[1] = 7
    c.old = c.call("fwd")["logprob"].astype(np.float32)               # ratio 1, the border on both sides
    got = c.call(how)
    for i in range(8):
        lp = got["logprob"][i]
        want = -c.adv[i] * (1 - np.exp(lp)) * c.w[i]
        assert abs(got["dz"][i, c.t[i]] - want) <= 1e-5 * abs(c.adv[i]) and got["loss"][i] == -c.adv[i]


@pytest.mark.parametrize("how", ["both", "step"])
@pytest.mark.parametrize("v", [300, 60000])
def test_masked_and_special_rows(how, v):
    c = Case(6, v, stp.STP_FP32, kl=0.2, ent=0.05)
    z = c.z.clone()
    z[:, v // 2:] = -INF                                              # a padded vocabulary
    z[3] = -INF                                                       # nothing at all
    z[4, 0] = NAN
    z[5, :] = torch.finfo(torch.float32).min                          # even, at the type's lowest value
    c = Case(6, v, stp.STP_FP32, kl=0.2, ent=0.05, z=z)
    c.t[:] = [3, -1, v - 1, 5, 6, 7]                                  # row 2: a token that cannot be
    got = c.call(how)
    assert c.status == stp.STP_OK
    assert got["logprob"][2] == -INF and (got["dz"][2] == 0).all() and got["kl"][2] == INF and got["loss"][2] == INF
    assert got["logprob"][3] == got["lse"][3] == -INF and got["entropy"][3] == 0 and (got["dz"][3] == 0).all()
    assert np.isnan(got["loss"][4]) and np.isnan(got["dz"][4]).any()
    assert abs(got["logprob"][5] + np.log(v)) <= 1e-4
    assert (got["dz"][0, v // 2:] == 0).all()
    for i in (1, 2, 3, 4, 5):
        c.t[i] = -1
    c.check({k: np.concatenate((x[:1], np.zeros_like(x[1:]))) for k, x in got.items()})


def test_step_at_large_logits_follows_the_differences():
    z = torch.randn(4, 700, generator=torch.Generator().manual_seed(2))
    c = Case(4, 700, stp.STP_FP32, kl=None, ent=0.0, z=(z * 2.0).round() / 8)     # exact after the shift
    far = Case(4, 700, stp.STP_FP32, kl=None, ent=0.0, z=(z * 2.0).round() / 8 + 1e6)
    a, b = c.call("step"), far.call("step")
    assert np.array_equal(a["logprob"], b["logprob"]) and np.array_equal(a["dz"], b["dz"])


@pytest.mark.parametrize("n", [7, 5000])
@pytest.mark.parametrize("how", ["fwd", "both", "step"])
def test_a_target_past_the_vocabulary(n, how):
    c = Case(n, 40, stp.STP_BF16)
    c.t[n - 1] = 40
    got = c.call(how)
    assert c.status == stp.STP_EDEVICE
    assert np.isnan(got["loss"][n - 1]) and np.isnan(got["logprob"][n - 1])
    if how != "fwd":
        assert (got["dz"][n - 1] == 0).all()
    c.t[n - 1] = -1
    got = {k: np.concatenate((x[:-1], np.zeros_like(x[-1:]))) for k, x in got.items()}
    c.check(got, stp.STP_EDEVICE)
    c.check(c.call(how))                                              # the word is cleared


def test_no_rows_null_kl_and_repeat():
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    stp.stp_policy_fwd(stp.policy_desc(0, 8), *[None] * 10, ws)
    assert stp.stp_device_status(ws) == stp.STP_OK
    c = Case(9, 30000, stp.STP_BF16)
    a, b = c.call("step"), c.call("step")
    assert all(np.array_equal(a[k], b[k]) for k in a)
    out = [torch.empty(9, device="cuda") for _ in range(4)]
    stp.stp_policy_fwd(c.desc, *c.given(), *out, None, ws)
    assert np.array_equal(out[0].double().cpu().numpy(), a["loss"])


def test_captured_and_on_another_stream():
    c = Case(20, 3000, stp.STP_BF16)
    want = c.call("step")
    side = torch.cuda.Stream()
    got = c.call("step", stream=side)
    assert all(np.array_equal(want[k], got[k]) for k in want)
    out = [torch.full((20,), NAN, device="cuda") for _ in NAMES]
    given, w, dz = c.given(), torch.from_numpy(c.w).cuda(), torch.full_like(c.z, NAN)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        stp.stp_policy_step(c.desc, *given, w, *out, dz, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(dz.double().cpu().numpy(), want["dz"]) and np.array_equal(out[0].double().cpu().numpy(), want["loss"])


@pytest.mark.parametrize("how", ["fwd", "both", "step"])
@pytest.mark.parametrize("n,v,dtype", [(1300, 513, stp.STP_BF16), (1300, 4096, stp.STP_FP32), (1217, 700, stp.STP_FP32), (9, 512, stp.STP_BF16),
                                       (40, 31, stp.STP_FP32), (700, 9000, stp.STP_BF16), (1216, 8192, stp.STP_BF16)])
def test_rows_of_a_warp_and_of_a_block(n, v, dtype, how):
    # both sides of the rules on sizes: short rows, many and few of them
    c = Case(n, v, dtype, scale=0.8)
    a = c.call(how)
    c.check(a)
    if how != "fwd":
        b = c.call(how, into=c.z)
        assert all(np.array_equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("n", [6, 1300])
@pytest.mark.parametrize("how", ["both", "step"])
def test_short_rows_strided_with_special_values(how, n):
    v = 300
    c = Case(n, v, stp.STP_BF16, stride=v + 3, offset=1)
    c.z[0, v // 2:] = -INF
    c.z[3] = -INF
    c.z[4, 7] = NAN
    c.z[5] = torch.finfo(torch.bfloat16).min
    c.t[:6] = [3, -1, 5, 6, 7, 8]
    between = c.z.as_strided((n - 1, 3), (v + 3, 1), c.z.storage_offset() + v).clone()
    want = {k: x.copy() for k, x in c.call(how).items()}
    assert want["logprob"][3] == -INF and (want["dz"][3] == 0).all() and want["entropy"][3] == 0
    assert np.isnan(want["loss"][4]) and np.isnan(want["dz"][4]).any() and (want["dz"][0, v // 2:] == 0).all()
    assert abs(want["logprob"][5] + np.log(v)) <= 1e-4 or how == "both"
    got = c.call(how, into=c.z)
    assert all(np.array_equal(want[k], got[k], equal_nan=True) for k in want)
    assert torch.equal(c.z.as_strided((n - 1, 3), (v + 3, 1), c.z.storage_offset() + v), between)
