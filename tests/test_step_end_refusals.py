"""What the policy loss, the embedding and the 8-bit checkpoint refuse.  No GPU
is touched: every call here ends in the library's own checks."""
import pytest

from sft_trie_build_gb300 import stp

A = 1 << 20          # an address no call may read: every one below is refused first


def refused(status, f, *args):
    with pytest.raises(stp.StpError) as e:
        f(*args, **({} if f.__name__.endswith("_size") else {"stream": 0}))
    assert e.value.status == status, e.value
    assert str(e.value)


def test_policy(stp_lib):
    d = stp.policy_desc
    fwd, bwd, step = stp.stp_policy_fwd, stp.stp_policy_bwd, stp.stp_policy_step
    nan = float("nan")
    for status, bad in ((stp.STP_EINVAL, d(-1, 8)), (stp.STP_EUNSUPPORTED, d(1, 0)), (stp.STP_EUNSUPPORTED, d(1, (1 << 24) + 1)),
                        (stp.STP_EINVAL, d(1, 8, stride=7)), (stp.STP_EUNSUPPORTED, d(1, 8, 9)), (stp.STP_EINVAL, d(1, 8, scale=0.0)),
                        (stp.STP_EINVAL, d(1, 8, scale=nan)), (stp.STP_EINVAL, d(1, 8, clip_low=-0.1)),
                        (stp.STP_EINVAL, d(1, 8, clip_low=1.5)), (stp.STP_EINVAL, d(1, 8, clip_high=nan)),
                        (stp.STP_EINVAL, d(1, 8, kl_coef=-1.0)), (stp.STP_EINVAL, d(1, 8, entropy_coef=nan))):
        refused(status, stp.stp_policy_workspace_size, bad)
        refused(status, fwd, bad, *[A] * 11)
        refused(status, bwd, bad, *[A] * 10)
        refused(status, step, bad, *[A] * 13)
    good = d(4, 8)
    for at in (0, 1, 2, 4, 5, 6, 7, 8, 10):          # all but ref_logprob and kl
        refused(stp.STP_EINVAL, fwd, good, *[None if i == at else A for i in range(11)])
    for at in (0, 1, 2, 4, 5, 6, 7, 8, 9):
        refused(stp.STP_EINVAL, bwd, good, *[None if i == at else A for i in range(10)])
    for at in (0, 1, 2, 4, 5, 6, 7, 8, 9, 11, 12):
        refused(stp.STP_EINVAL, step, good, *[None if i == at else A for i in range(13)])
    refused(stp.STP_EINVAL, fwd, d(4, 8, kl_coef=0.1), A, A, A, None, *[A] * 7)       # a KL term without a reference
    refused(stp.STP_EINVAL, fwd, good, A + 1, *[A] * 10)                            # off its type
    refused(stp.STP_EINVAL, fwd, good, *[A] * 10, A + 16)                           # workspace
    refused(stp.STP_EINVAL, bwd, good, *[A] * 9, A + 1)
    assert stp.stp_policy_workspace_size(good) == 256
    bwd(d(0, 8), *[None] * 10, stream=0)                                            # no row: nothing to do


def test_embed(stp_lib):
    d = stp.embed_desc
    fwd, bwd = stp.stp_embed_fwd, stp.stp_embed_bwd
    for status, bad in ((stp.STP_EINVAL, d(-1, 8, 8)), (stp.STP_EUNSUPPORTED, d((1 << 28) + 1, 8, 8)),
                        (stp.STP_EUNSUPPORTED, d(1, 0, 8)), (stp.STP_EUNSUPPORTED, d(1, (1 << 24) + 1, 8)),
                        (stp.STP_EUNSUPPORTED, d(1, 8, 0)), (stp.STP_EUNSUPPORTED, d(1, 8, 12)),
                        (stp.STP_EUNSUPPORTED, d(1, 8, 65544)), (stp.STP_EUNSUPPORTED, d(1, 8, 6, stp.STP_FP32)),
                        (stp.STP_EUNSUPPORTED, d(1, 8, 8, 5)), (stp.STP_EINVAL, d(1, 8, 16, stride=8)),
                        (stp.STP_EINVAL, d(1, 8, 16, stride=20)), (stp.STP_EINVAL, d(1, 8, 16, scale=float("nan"))),
                        (stp.STP_EINVAL, d(1, 8, 16, scale=2e6))):
        refused(status, stp.stp_embed_workspace_size, bad)
        refused(status, fwd, bad, A, A, A, A)
        refused(status, bwd, bad, A, A, 0, A, A)
    good = d(4, 8, 16)
    for at in range(4):
        refused(stp.STP_EINVAL, fwd, good, *[None if i == at else A for i in range(4)])
        refused(stp.STP_EINVAL, bwd, good, *[x for i, x in enumerate((A, A, A, A)) if i < 2 for x in [None if i == at else A]],
                0, *[None if i == at else A for i in (2, 3)])
    refused(stp.STP_EINVAL, fwd, good, A + 8, A, A, A)
    refused(stp.STP_EINVAL, fwd, good, A, A, A + 8, A)
    refused(stp.STP_EINVAL, fwd, good, A, A, A, A + 16)
    refused(stp.STP_EINVAL, bwd, good, A + 8, A, 0, A, A)
    refused(stp.STP_EINVAL, bwd, good, A, A, 0, A + 4, A)
    refused(stp.STP_EINVAL, bwd, good, A, A, 1, A, A + 16)
    assert stp.stp_embed_workspace_size(good) >= 256 + 2 * 4 * 8


def test_ckpt(stp_lib):
    d = stp.ckpt_desc
    for status, bad in ((stp.STP_EINVAL, d(-1, 8)), (stp.STP_EUNSUPPORTED, d((1 << 24) + 1, 8)), (stp.STP_EUNSUPPORTED, d(1, 0)),
                        (stp.STP_EUNSUPPORTED, d(1, 65537)), (stp.STP_EUNSUPPORTED, d(1, 8, 5)), (stp.STP_EINVAL, d(1, 8, stride=7))):
        refused(status, stp.stp_ckpt_size, bad)
        refused(status, stp.stp_ckpt_save, bad, A, A)
        refused(status, stp.stp_ckpt_load, bad, A, A)
        refused(status, stp.stp_ckpt_wgrad_workspace_size, bad, 8)
        refused(status, stp.stp_ckpt_wgrad, bad, 8, A, A, 8, 0, A, A)
    good = d(4, 8)
    for f in (stp.stp_ckpt_save, stp.stp_ckpt_load):
        refused(stp.STP_EINVAL, f, good, None, A)
        refused(stp.STP_EINVAL, f, good, A, None)
    refused(stp.STP_EINVAL, stp.stp_ckpt_save, good, A + 1, A)
    refused(stp.STP_EINVAL, stp.stp_ckpt_save, good, A, A + 16)
    refused(stp.STP_EINVAL, stp.stp_ckpt_load, good, A + 16, A)
    refused(stp.STP_EINVAL, stp.stp_ckpt_load, d(4, 8, stp.STP_FP32), A, A + 2)
    assert stp.stp_ckpt_size(d(129, 33)) == (4 * 4352 + 255) // 256 * 256 and stp.stp_ckpt_size(d(0, 33)) == 0
    stp.stp_ckpt_save(d(0, 8), None, None, stream=0)                                # no token: nothing to do


def test_wgrad(stp_lib):
    d = stp.ckpt_desc(4, 8)
    f = stp.stp_ckpt_wgrad
    for cols in (0, -1, (1 << 20) + 1):
        refused(stp.STP_EUNSUPPORTED, stp.stp_ckpt_wgrad_workspace_size, d, cols)
        refused(stp.STP_EUNSUPPORTED, f, d, cols, A, A, 8, 0, A, A)
    refused(stp.STP_EINVAL, f, d, 8, None, A, 8, 0, A, A)
    refused(stp.STP_EINVAL, f, d, 8, A, None, 8, 0, A, A)
    refused(stp.STP_EINVAL, f, d, 8, A, A, 8, 0, None, A)
    refused(stp.STP_EINVAL, f, d, 8, A, A, 8, 0, A, None)
    refused(stp.STP_EINVAL, f, d, 16, A, A, 8, 0, A, A)                             # rows shorter than cols
    refused(stp.STP_EINVAL, f, d, 9, A, A, 9, 0, A, A)                              # not whole 16 bytes
    refused(stp.STP_EINVAL, f, d, 8, A + 16, A, 8, 0, A, A)
    refused(stp.STP_EINVAL, f, d, 8, A, A + 8, 8, 0, A, A)
    refused(stp.STP_EINVAL, f, d, 8, A, A, 8, 0, A + 2, A)
    refused(stp.STP_EINVAL, f, d, 8, A, A, 8, 0, A, A + 16)
