"""Policy gradients with large weights and entropy coefficients beside logits
that are masked: what has probability 0 has a gradient of 0, whatever the
other factors are (stp_policy_bwd, stp_policy_step).  Bounds as in
tests/test_gpu_policy.py."""
import numpy as np
import pytest
import torch

from sft_trie_build_gb300 import stp
from test_gpu_policy import DT, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low", [-float("inf"), None])                # None: the type's lowest value
@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("how", ["both", "step"])
@pytest.mark.parametrize("v", [301, 2001, 60001])                     # a row is a warp's, a block's, several blocks'
def test_masked_logits_have_no_gradient(v, how, dtype, low):
    c = Case(5, v, dtype, kl=0.2, ent=1000.0)
    z = c.z.clone()
    z[:, 7] = 20.0                                                    # nearly all of the weight
    z[:, v // 2:] = torch.finfo(DT[dtype]).min if low is None else low
    c = Case(5, v, dtype, kl=0.2, ent=1000.0, z=z)
    c.t[:] = [7, -1, 8, 7, v // 2 - 1]
    c.w[:] = 1e6                                                      # 1e9 ln p passes float32's range where ln p is held at -1e30
    got = c.call(how)
    assert (got["dz"][:, v // 2:] == 0).all()
    if low is not None:
        c.check(got)                                                  # whose bound counts finite logits, the lowest one too
    else:
        assert np.isfinite(got["dz"]).all()


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("how", ["both", "step"])
@pytest.mark.parametrize("ent", [0.0, 0.1])
@pytest.mark.parametrize("v", [301, 2001, 60001])
def test_factors_beyond_float32(v, ent, how, dtype):
    c = Case(5, v, dtype, kl=0.2, ent=ent)
    z = c.z.clone()
    z[:, v // 2:] = -float("inf")
    c = Case(5, v, dtype, kl=0.2, ent=ent, z=z)
    c.t[:] = [3, -1, 4, 5, 6]
    lp = c.call("fwd")["logprob"].astype(np.float32)
    c.old, c.ref = lp - np.float32(0.01), lp + np.float32(0.01)
    c.adv[:] = [-1, 1, -1, 1, -1]
    c.old[0] = -200                                                   # a ratio above e^88 that is not clipped,
    c.old[3] = -200                                                   # one that is,
    c.ref[4] = lp[4] + 100                                            # and a token that the reference holds for far likelier
    got = c.call(how)
    assert c.status == stp.STP_OK and np.isfinite(got["dz"]).all() and (got["dz"][:, v // 2:] == 0).all()
    assert got["loss"][0] == got["loss"][4] == got["kl"][4] == np.inf
    top = float(torch.finfo(torch.bfloat16).max)
    assert got["dz"][0, 3] > 0.5 * top and got["dz"][4, 6] < -0.5 * top    # the way out, as far as there are numbers
    c.t[[0, 4]] = -1
    c.check({k: np.where((np.arange(5) % 4 == 0).reshape((5,) + (1,) * (x.ndim - 1)), 0, x) for k, x in got.items()})
