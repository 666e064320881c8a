"""Forms of the policy step that other sizes do not reach, and the digits of
likely tokens (stp_policy_step, stp_policy_fwd).

Likely tokens.  With scale the float32 number next to ln 2, scale log2 e rounds
to 1, and whole logits at most 20 below the target's give exponentials that are powers of two: all
sums are exact in any order.  So the log-probability is off by the
exponentials' 2^-22 and the logarithm's last place: 2^-21 of itself; and 1 - p
by the rounding of 1 / s and its product: 2^-23.  The scale's own distance from
ln 2 is 2^-28 of it, 20 2^-28 of a probability other than the target's.
kl = exp(x) - x - 1 at x = ref - lp, off by 2^-21 |lp| + 2^-24 |x|: that times
its derivative exp(x) - 1, and 2^-20 of itself for the series or, beyond 1/2,
for the difference of two numbers at most 8 times as large.  Adding a whole
number to every logit changes nothing.
"""
import numpy as np
import pytest
import torch

from oracle import policy as OP
from sft_trie_build_gb300 import stp
from test_gpu_policy import DT, NAMES, Case

pytestmark = pytest.mark.gpu
LN2 = float(np.float32(np.log(2)))


@pytest.mark.parametrize("v,dtype", [(60000, stp.STP_BF16), (60013, stp.STP_BF16), (30000, stp.STP_FP32), (30007, stp.STP_FP32)])
def test_a_step_with_a_block_to_a_row_above_100_kb(v, dtype):
    # 608 rows and more are a block's each; the other rows have no token, so that few are compared
    n, live = 700, [0, 1, 77, 350, 698, 699]
    g = torch.Generator(device="cuda").manual_seed(v)
    stride = v + 3
    z = (torch.randn(n * stride, generator=g, device="cuda") * 3).to(DT[dtype]).as_strided((n, v), (stride, 1))
    c = Case(len(live), v, dtype, z=z[live])
    c.t[:] = [0, v - 1, -1, 5, v // 2, v - 2]

    def wide(x, fill):
        out = torch.full((n,), fill, dtype=torch.from_numpy(x).dtype, device="cuda")
        out[live] = torch.from_numpy(x).cuda()
        return out

    given = wide(c.t, -1), wide(c.old, 0), wide(c.ref, 0), wide(c.adv, 0), wide(c.w, 1)
    desc = stp.policy_desc(n, v, dtype, c.scale, c.low, c.high, c.kl, c.ent, stride)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    first = None
    for into in (torch.full((n * stride,), float("nan"), dtype=z.dtype, device="cuda").as_strided((n, v), (stride, 1)), z):
        out = {k: torch.full((n,), float("nan"), device="cuda") for k in NAMES}
        stp.stp_policy_step(desc, z, *given, *out.values(), into, ws)
        c.status = stp.stp_device_status(ws)
        got = {k: x[live].double().cpu().numpy() for k, x in {**out, "dz": into}.items()}
        c.check(got)
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        rest[live] = False
        assert not into[rest].any() and not out["loss"][rest].any()
        if first is not None:
            assert all(np.array_equal(first[k], got[k]) for k in got)
        first = got


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("shift", [0, -100])
@pytest.mark.parametrize("n,v", [(24, 500), (24, 3001), (24, 40000), (1300, 3001)])    # a row is a warp's, a block's, several blocks'
def test_likely_tokens_keep_their_digits(n, v, shift, dtype):
    rng = np.random.default_rng(v + n)
    z = -rng.integers(17, 21, (n, v)).astype(np.float64)
    t = rng.integers(0, v, n)
    z[np.arange(n), t] = 0
    scale = LN2
    lp = np.array([-np.log1p((np.exp(np.delete(r, k) * scale)).sum()) for r, k in zip(z, t)])
    p = np.exp(lp)
    assert (p < 1 - 1e-4).all() and (p > 0.7).all()
    old = np.zeros(n, np.float32)
    ref = (lp * rng.choice([1.5, 0.5, 1.001, 300.0], n)).astype(np.float32)
    adv = np.ones(n, np.float32)
    desc = stp.policy_desc(n, v, dtype, scale, 1.0, 1.0, 0.0, 0.0)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    logits = dev(z + shift).to(DT[dtype])
    assert np.array_equal(logits.double().cpu().numpy(), z + shift)
    out = {k: torch.full((n,), float("nan"), device="cuda") for k in NAMES}
    ws, dz = torch.empty(256, dtype=torch.uint8, device="cuda"), torch.full_like(logits, float("nan"))
    stp.stp_policy_step(desc, logits, dev(t.astype(np.int32)), dev(old), dev(ref), dev(adv), dev(adv), *out.values(), dz, ws)
    assert stp.stp_device_status(ws) == stp.STP_OK
    got = {k: x.double().cpu().numpy() for k, x in out.items()}
    off = 20 * 2.0 ** -28 * (1 - p)
    assert (np.abs(got["logprob"] - lp) <= 2.0 ** -21 * np.abs(lp) + off).all()
    x = ref.astype(np.float64) - lp
    kl = np.expm1(x) - x
    assert (np.abs(x) <= 300).all()
    assert (np.abs(got["kl"] - kl) <= np.maximum(np.abs(np.expm1(x)), 1e-300) * (2.0 ** -21 * np.abs(lp) + 2.0 ** -24 * np.abs(x) + off)
            + 2.0 ** -20 * kl).all()
    # the ratio is exp(lp): its own rounding, 2^-22, and that of its exponent; then 1 - p, and one rounding to the type
    want = -p * (1 - p) * scale
    u = torch.finfo(DT[dtype]).eps / 2
    tol = u * np.abs(want) + (1 + u) * (2.0 ** -21 * np.abs(want) + scale * (2.0 ** -22 + off))
    assert (np.abs(dz.double().cpu().numpy()[np.arange(n), t] - want) <= tol).all()
    assert OP.row(z[0] + shift, t[0], 0.0, float(ref[0]), 1.0, 1.0, 1.0, 0.0, 0.0, scale)[4] == pytest.approx(kl[0], rel=1e-6, abs=1e-12)
