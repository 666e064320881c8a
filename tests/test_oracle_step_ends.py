"""The oracles of the policy loss, the embedding and the 8-bit checkpoint on
the CPU: closed forms, finite differences, exhaustive rounding."""
import numpy as np
import pytest
import torch

from oracle import ckpt as OC
from oracle import embed as OE
from oracle import policy as OP


@pytest.mark.parametrize("adv,move", [(1.5, 0.1), (1.5, 0.5), (-0.7, -0.1), (-0.7, -0.5), (1.5, -0.9), (-0.7, 0.9), (0.0, 0.3)])
@pytest.mark.parametrize("kl_coef,entropy_coef", [(0.0, 0.0), (0.3, 0.0), (0.2, 0.5)])
def test_policy_gradient_by_differences(adv, move, kl_coef, entropy_coef):
    rng = np.random.default_rng(3)
    z = rng.standard_normal(7) * 2
    _, lp, *_ = OP.row(z, 4, 0.0, None, 0.0, 0.2, 0.28, 0.0, 0.0, 0.8)
    args = (4, lp - move, lp + 0.4, adv, 0.2, 0.28, kl_coef, entropy_coef, 0.8)
    grad = OP.row(z, *args)[-1]
    for v in range(7):
        step = np.zeros(7)
        step[v] = 1e-6
        diff = (OP.row(z + step, *args)[0] - OP.row(z - step, *args)[0]) / 2e-6
        # the differences' error: third derivatives times 1e-12, and 1e-16 / 1e-6 of the values
        assert abs(diff - grad[v]) <= 1e-8


def test_policy_closed_forms():
    z = np.log(np.array([1.0, 2.0, 5.0]))
    loss, lp, ent, lse, kl, _ = OP.row(z, 1, np.log(0.25), np.log(0.25), 2.0, 0.2, 0.2, 1.0, 0.0)
    # the probability is 1/4 under all three policies: ratio 1, no divergence
    assert abs(lp - np.log(0.25)) < 1e-15 and abs(loss + 2) < 1e-15 and abs(kl) < 1e-15 and abs(lse - np.log(8)) < 1e-15
    assert OP.terms(0.0, 0.0, -1.0, None, 1.0, 0.2, 0.3, 0.0, 0.0) == (-1.3, 0.0, 0.0)      # clipped from above
    assert OP.terms(-1.0, 0.0, 0.0, None, -1.0, 0.2, 0.3, 0.0, 0.0)[0] == 0.8               # and from below
    loss, kl, g = OP.terms(-1.0, 2.0, -1.0, 0.0, 0.0, 0.2, 0.3, 0.5, 0.25)
    assert abs(kl - (np.e - 2)) < 1e-15 and abs(loss - 0.5 * (np.e - 2) + 0.5) < 1e-15 and abs(g + 0.5 * (np.e - 1)) < 1e-15


def test_embed():
    table = np.arange(12.0).reshape(4, 3)
    assert OE.fwd(table, [2, -1, 0, 9], 2.0).tolist() == [[12, 14, 16], [0, 0, 0], [0, 2, 4], [0, 0, 0]]
    grad, size, count = OE.bwd(np.array([[1.0, -2.0], [3.0, 4.0], [5.0, 6.0]]), [1, -1, 1], 3, -0.5)
    assert grad.tolist() == [[0, 0], [-3, -2], [0, 0]] and size.tolist() == [[0, 0], [3, 4], [0, 0]] and count.tolist() == [0, 2, 0]


def test_e4m3_is_the_nearest_of_all_numbers():
    every = np.unique(torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    every = every[np.isfinite(every)]
    mids = (every[1:] + every[:-1]) / 2
    for v in (every, mids, np.nextafter(mids, 1e9), np.nextafter(mids, -1e9), np.random.default_rng(0).uniform(-448, 448, 5000)):
        near = np.abs(v[:, None] - every[None]).min(1)
        got = OC.e4m3(v)
        assert np.isin(got, every).all() and (np.abs(got - v) == near).all()
    want = torch.from_numpy(mids.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()   # ties
    assert np.array_equal(OC.e4m3(mids), want)


def test_scales():
    x = np.zeros((9, 40), np.float32)
    tops = np.array([448, 449, 3.5, 3.5000002, 0.4375, 3e38, 1e-40, 0, np.inf], np.float32)
    x[:, 3] = tops
    x[4, 35] = np.nan
    s = OC.scales(x)
    want = [1, 2, 2.0 ** -7, 2.0 ** -6, 2.0 ** -10, 2.0 ** 120, 2.0 ** -117, 2.0 ** -117, np.nan]
    assert np.array_equal(s[:, 0], want, equal_nan=True)
    assert np.isnan(s[4, 1]) and s[0, 1] == 2.0 ** -117
    k = OC.keep(x)
    assert np.isnan(k[8, :32]).all() and (k[8, 32:] == 0).all() and np.isnan(k[4, 32:]).all() and k[4, 3] == tops[4]
    live = np.isfinite(k)
    assert (np.abs(k - x)[live] <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * np.repeat(s, 32, 1)[:, :40])[live]).all()
