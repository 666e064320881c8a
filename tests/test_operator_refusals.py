"""What q/k norm with rotation, windowed attention, token statistics and
distillation refuse, and the host count of windowed tile pairs.  No GPU is
touched: every call here ends in the library's own checks."""
import numpy as np
import pytest

from oracle import pack as OP
from oracle import window as OW
from sft_trie_build_gb300 import stp
from sft_trie_build_gb300 import workloads as W

A = 1 << 20          # an address no call may read: every one below is refused first


def refused(status, f, *args):
    with pytest.raises(stp.StpError) as e:
        f(*args)
    assert e.value.status == status, e.value
    assert str(e.value)


def _fwd(desc, q=A, k=A, freq=np.ones(512), pos=A, qo=A, ko=A):
    stp.stp_qk_norm_rope_fwd(desc, q, k, None, None, freq, pos, qo, ko, stream=0)


def test_qk_descriptors(stp_lib):
    d = stp.qk_desc
    for bad in (d(4, 0, 1), d(4, 1, 0), d(4, 1, 5000), d(4, 1, 1, 24), d(4, 1, 1, 528), d(4, 1, 1, 0),
                d(4, 1, 1, 64, 72), d(4, 1, 1, 64, 24), d(4, 1, 1, 64, -16), d(4, 1, 1, dtype=7)):
        refused(stp.STP_EUNSUPPORTED, _fwd, bad)
        refused(stp.STP_EUNSUPPORTED, stp.stp_qk_norm_rope_workspace_size, bad)
    for bad in (d(-1, 1, 1), d(4, 1, 1, eps=-1.0), d(4, 1, 1, eps=float("nan")), d(4, 2, 1, q_stride=255),
                d(4, 2, 1, q_stride=257), d(4, 1, 2, k_stride=128), d(4, 1, 1, dtype=stp.STP_FP32, k_stride=130),
                stp.QkDesc(4, 1, 1, 128, 128, 2, 0, 1e-6, 128, 128)):
        refused(stp.STP_EINVAL, _fwd, bad)


def test_qk_arguments(stp_lib):
    d = stp.qk_desc(4, 1, 1)
    refused(stp.STP_EINVAL, _fwd, d, None)
    refused(stp.STP_EINVAL, _fwd, d, A + 8)
    refused(stp.STP_EINVAL, _fwd, d, A, A, None)
    refused(stp.STP_EINVAL, _fwd, d, A, A, np.full(64, np.inf))
    refused(stp.STP_EINVAL, _fwd, d, A, A, np.ones(64), None)
    refused(stp.STP_EINVAL, _fwd, d, A, A, np.ones(64), A, A + 2)
    with pytest.raises(ValueError):
        _fwd(d, A, A, np.ones(63))
    _fwd(stp.qk_desc(0, 1, 1), None, None, np.ones(64), None, None, None)      # no token: nothing to do
    bwd = lambda *a: stp.stp_qk_norm_rope_bwd(d, A, A, None, None, np.ones(64), A, *a, stream=0)  # noqa: E731
    refused(stp.STP_EINVAL, bwd, A, A, A, A, None, A, A)
    refused(stp.STP_EINVAL, bwd, A, A, A, A, A, A, None)
    refused(stp.STP_EINVAL, bwd, A, A, A, A, A, A, A + 16)
    refused(stp.STP_EINVAL, bwd, A + 8, A, A, A, A, A, A)
    assert stp.stp_qk_norm_rope_workspace_size(d) >= 128 * 4


def test_window_arguments(stp_lib):
    d = stp.Desc(1, 256, 2, 1, 128)
    cls = lambda w, m, se=A, pos=A, meta=A, d=d: stp.stp_classify_window(d, w, m, se, pos, meta, stream=0)  # noqa: E731
    for w, m in ((0, 0), (-5, 0), (4, -1)):
        refused(stp.STP_EINVAL, cls, w, m)
        refused(stp.STP_EINVAL, lambda: stp.stp_attn_window_fwd(d, w, m, *[A] * 9, stream=0))
        refused(stp.STP_EINVAL, lambda: stp.stp_attn_window_bwd(d, w, m, *[A] * 13, stream=0))
        refused(stp.STP_EINVAL, stp.stp_count_window_tile_pairs, np.zeros((0, 128)), np.zeros((0, 128)), w, m)
    refused(stp.STP_EINVAL, cls, 4, 0, None)
    refused(stp.STP_EINVAL, cls, 4, 0, A, None)
    refused(stp.STP_EINVAL, cls, 4, 0, A, A + 4)
    refused(stp.STP_EINVAL, cls, 4, 0, A, A, A + 128)
    refused(stp.STP_EUNSUPPORTED, cls, 4, 0, A, A, A, stp.Desc(1, 200, 2, 1, 128))
    refused(stp.STP_EINVAL, lambda: stp.stp_attn_window_fwd(d, 4, 0, A, A, A, A, None, A, A, A, A, stream=0))
    refused(stp.STP_EINVAL, lambda: stp.stp_attn_window_fwd(d, 4, 0, A, A, A, A, A + 4, A, A, A, A, stream=0))
    refused(stp.STP_EINVAL, lambda: stp.stp_attn_window_bwd(d, 4, 0, *[A] * 7, None, *[A] * 5, stream=0))


def test_count_window_tile_pairs(stp_lib):
    se, pos = np.full((1, 1024), 1023, np.int32), np.arange(1024, dtype=np.int32)[None]     # one sequence
    count = stp.stp_count_window_tile_pairs
    assert count(se, pos, 1, 0) == 8                       # the diagonal
    assert count(se, pos, 2, 0) == 8 + 7
    assert count(se, pos, 129, 0) == 8 + 7 and count(se, pos, 130, 0) == 8 + 7 + 6
    assert count(se, pos, 1, 1) == 8 + 7                   # and the first tile from everywhere
    assert count(se, pos, 1, 129) == 8 + 7 + 6
    assert count(se, pos, 2 ** 31 - 1, 0) == stp.stp_count_tile_pairs(se) == 36
    for bad in (-1, 1 << 30):
        p = pos.copy()
        p[0, 77] = bad
        refused(stp.STP_EINVAL, count, se, p, 4, 0)
    s = se.copy()
    s[0, 5] = 4
    refused(stp.STP_EINVAL, count, s, pos, 4, 0)
    with pytest.raises(ValueError):
        count(se, pos[:, :512], 4, 0)


@pytest.mark.parametrize("seed", range(6))
def test_counted_pairs_cover_the_visible_ones(stp_lib, seed):
    b = W.random_forest(seed, n_roots=4, max_depth=3, len_lo=5, len_hi=90, row_len=1024, min_shared=8)
    plan = OP.pack(b.seqs, b.trainable, b.row_len, b.min_shared)
    every = stp.stp_count_tile_pairs(plan.subtree_end)
    for window, sinks in ((1, 0), (30, 4), (200, 0)):
        m = OW.mask(plan, window, sinks)
        need = m.reshape(len(m), 8, 128, 8, 128).any((2, 4)).sum()
        assert need <= stp.stp_count_window_tile_pairs(plan.subtree_end, plan.position_ids, window, sinks) <= every


def _stats(desc, z=A, t=A, ws=A, top=A):
    stp.stp_token_stats_fwd(desc, z, t, A, A, A, top, top, ws, stream=0)


def test_stats(stp_lib):
    d = stp.stats_desc
    for bad in (d(4, 0), d(4, (1 << 24) + 1), d(4, 100, 33), d(4, 100, -1), d(4, 100, dtype=3)):
        refused(stp.STP_EUNSUPPORTED, _stats, bad)
        refused(stp.STP_EUNSUPPORTED, stp.stp_token_stats_workspace_size, bad)
    for bad in (d(-1, 100), d(4, 100, stride=99), d(4, 100, scale=0.0), d(4, 100, scale=float("nan")), d(4, 100, scale=-1.0)):
        refused(stp.STP_EINVAL, _stats, bad)
    ok = d(4, 100, 2)
    refused(stp.STP_EINVAL, _stats, ok, None)
    refused(stp.STP_EINVAL, _stats, ok, A, None)
    refused(stp.STP_EINVAL, _stats, ok, A, A, None)
    refused(stp.STP_EINVAL, _stats, ok, A, A, A + 4)
    refused(stp.STP_EINVAL, _stats, ok, A + 1)
    refused(stp.STP_EINVAL, _stats, ok, A, A, A, None)
    bwd = lambda *a: stp.stp_token_stats_bwd(ok, *a, stream=0)  # noqa: E731
    refused(stp.STP_EINVAL, bwd, A, A, None, A, A, A, A)
    refused(stp.STP_EINVAL, bwd, A, A, A, None, A, A, A)       # an entropy gradient without the entropy
    refused(stp.STP_EINVAL, bwd, A, A, A, A, A, A, A + 1)
    stp.stp_token_stats_bwd(d(0, 100), *[None] * 7, stream=0)


def test_distill(stp_lib):
    d = stp.distill_desc
    fwd = lambda desc, z=A, i=A, t=A, ws=A: stp.stp_distill_fwd(desc, z, i, t, None, A, A, ws, stream=0)  # noqa: E731
    for bad in (d(4, 0, 1), d(4, 100, 0), d(4, 100, 257), d(4, 100, 4, dtype=2)):
        refused(stp.STP_EUNSUPPORTED, fwd, bad)
        refused(stp.STP_EUNSUPPORTED, stp.stp_distill_workspace_size, bad)
    for bad in (d(-1, 100, 4), d(4, 100, 4, stride=1), d(4, 100, 4, scale=0.0)):
        refused(stp.STP_EINVAL, fwd, bad)
    ok = d(4, 100, 4, stp.STP_FP32)
    refused(stp.STP_EINVAL, fwd, ok, None)
    refused(stp.STP_EINVAL, fwd, ok, A + 2)
    refused(stp.STP_EINVAL, fwd, ok, A, None)
    refused(stp.STP_EINVAL, fwd, ok, A, A, None)
    refused(stp.STP_EINVAL, fwd, ok, A, A, A, None)
    refused(stp.STP_EINVAL, fwd, ok, A, A, A, A + 8)
    refused(stp.STP_EINVAL, lambda: stp.stp_distill_bwd(ok, A, A, A, None, None, A, A, stream=0))
    refused(stp.STP_EINVAL, lambda: stp.stp_distill_bwd(ok, A, A, A, None, A, None, A, stream=0))
    refused(stp.STP_EINVAL, lambda: stp.stp_distill_step(ok, A, A, A, None, A, A, A, None, A, stream=0))
    refused(stp.STP_EINVAL, lambda: stp.stp_distill_step(ok, A, A, A, None, A, A, A, A + 2, A, stream=0))
    stp.stp_distill_bwd(d(0, 100, 4), *[None] * 7, stream=0)
