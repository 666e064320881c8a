"""Pins of the oracles of q/k norm with rotation (oracle/qk.py), windowed tree
attention (oracle/window.py) and losses on logits (oracle/token_loss.py):
closed forms, packed rows against every sequence alone, and finite
differences."""
import numpy as np
import pytest

from oracle import pack as OP
from oracle import qk as OQ
from oracle import token_loss as OT
from oracle import window as OW
from oracle.attn import RowTree
from sft_trie_build_gb300 import workloads as W


def _diff(f, x, eps=1e-6):
    """Central differences of f at x."""
    g = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


# ------------------------------------------------------------------ q/k norm and rotation

@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_norms_and_sees_distances_only(inter):
    rng = np.random.default_rng(0)
    f = 100.0 ** (-np.arange(4) / 4)
    q, k = rng.standard_normal((2, 1, 1, 8))
    w = np.ones(8)
    one = OQ.forward(q, w, [3], f, 8, inter)
    np.testing.assert_allclose((one ** 2).sum(), (q / np.sqrt((q * q).mean() + 1e-6)).__pow__(2).sum())
    dots = [(OQ.forward(q, w, [t + 5], f, 8, inter) * OQ.forward(k, w, [t], f, 8, inter)).sum() for t in (0, 17, 4000)]
    np.testing.assert_allclose(dots, dots[0])


def test_rotation_pairs_and_rest():
    x = np.array([3.0, 0, 0, 0, 0, 0, 4, 0]).reshape(1, 1, 8)
    n = x / np.sqrt(25 / 8)
    quarter = np.array([np.pi / 2, 0.0])
    half = OQ.forward(x, np.ones(8), [1], quarter, 4, False, 0.0)   # pairs (0, 2), (1, 3)
    np.testing.assert_allclose(half, np.array([0, 0, 3, 0, 0, 0, 4, 0]).reshape(1, 1, 8) * (n[0, 0, 0] / 3), atol=1e-12)
    inter = OQ.forward(x, np.ones(8), [1], quarter, 4, True, 0.0)   # pairs (0, 1), (2, 3)
    np.testing.assert_allclose(inter, np.array([0, 3, 0, 0, 0, 0, 4, 0]).reshape(1, 1, 8) * (n[0, 0, 0] / 3), atol=1e-12)


@pytest.mark.parametrize("rot,inter", [(8, False), (8, True), (4, False), (0, False)])
def test_qk_backward_against_differences(rot, inter):
    rng = np.random.default_rng(rot + inter)
    x, w, dy = rng.standard_normal((2, 3, 8)), rng.standard_normal(8), rng.standard_normal((2, 3, 8))
    pos, f = np.array([5, 11]), rng.random(rot // 2)
    dx, dw = OQ.backward(x, w, pos, f, rot, dy, inter, 1e-3)
    np.testing.assert_allclose(dx, _diff(lambda a: (OQ.forward(a, w, pos, f, rot, inter, 1e-3) * dy).sum(), x), atol=1e-8)
    np.testing.assert_allclose(dw, _diff(lambda a: (OQ.forward(x, a, pos, f, rot, inter, 1e-3) * dy).sum(), w), atol=1e-8)


# ------------------------------------------------------------------ windowed attention

@pytest.mark.parametrize("seed,window,sinks", [(0, 1, 0), (1, 7, 2), (2, 40, 4), (3, 1000, 0), (4, 5, 1000)])
def test_windowed_rows_equal_sequences_alone(seed, window, sinks):
    """Each sequence's outputs from its packed row equal windowed causal
    attention on the sequence alone."""
    b = W.random_forest(seed, n_roots=3, max_depth=3, len_lo=2, len_hi=30, row_len=256, min_shared=4, vocab=50)
    plan = OP.pack(b.seqs, b.trainable, b.row_len, b.min_shared)
    rng = np.random.default_rng(seed)
    E, P = rng.standard_normal((3, 50, 4)), rng.standard_normal((3, 256, 4))
    x = [E[c][plan.token_ids] + P[c][plan.position_ids] for c in range(3)]          # q, k, v by (token, position)
    got = OW.attention(OW.mask(plan, window, sinks), *(a[:, :, None] for a in x), 0.5)["o"].reshape(-1, 4)
    at = 0
    for seq in b.seqs:
        n = len(seq)
        q, k, v = (E[c][seq] + P[c][np.arange(n)] for c in range(3))
        i, j = np.arange(n)[:, None], np.arange(n)[None]
        s = np.where((j <= i) & ((i - j < window) | (j < sinks)), 0.5 * q @ k.T, -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        np.testing.assert_allclose(got[plan.gather_index[at:at + n]], p / p.sum(1, keepdims=True) @ v, atol=1e-12)
        at += n


def test_window_predicate_on_positions():
    """The mask along paths equals the predicate on subtree_end and position ids."""
    b = W.random_forest(9, n_roots=3, max_depth=3, len_lo=2, len_hi=40, row_len=512, min_shared=4)
    plan = OP.pack(b.seqs, b.trainable, b.row_len, b.min_shared)
    i, j = np.arange(512)[:, None], np.arange(512)[None]
    for window, sinks in ((1, 0), (9, 3), (64, 64)):
        for r, m in enumerate(OW.mask(plan, window, sinks)):
            se, pos = plan.subtree_end[r], plan.position_ids[r].astype(np.int64)
            near = (pos[:, None] - pos[None] < window) | (pos[None] < sinks)
            np.testing.assert_array_equal(m, (j <= i) & (se[None] >= i) & near)
    assert RowTree(plan, 0).used < 512      # pads were among them


def test_window_backward_against_differences():
    b = W.random_forest(2, n_roots=1, max_depth=2, len_lo=2, len_hi=5, row_len=24, min_shared=2)
    plan = OP.pack(b.seqs, b.trainable, b.row_len, b.min_shared)
    m = OW.mask(plan, 3, 1)[:1]
    rng = np.random.default_rng(0)
    q, do = rng.standard_normal((2, 1, 24, 2, 3))
    k, v = rng.standard_normal((2, 1, 24, 1, 3))
    r = OW.attention(m, q, k, v, 0.7, do)
    loss = lambda q, k, v: (OW.attention(m, q, k, v, 0.7)["o"] * do).sum()  # noqa: E731
    np.testing.assert_allclose(r["dq"], _diff(lambda x: loss(x, k, v), q), atol=1e-8)
    np.testing.assert_allclose(r["dk"], _diff(lambda x: loss(q, x, v), k), atol=1e-8)
    np.testing.assert_allclose(r["dv"], _diff(lambda x: loss(q, k, x), v), atol=1e-8)


# ------------------------------------------------------------------ logits

def test_stats_closed_forms():
    lp, ent, lse, ids, top = OT.stats_row(np.zeros(16), 3, 4)
    np.testing.assert_allclose([lp, ent, lse], [-np.log(16), np.log(16), np.log(16)])
    assert ids.tolist() == [0, 1, 2, 3]
    z = np.array([-np.inf, 2.0, -np.inf, 2.0])
    lp, ent, lse, ids, top = OT.stats_row(z, 0, 3)
    assert lp == -np.inf and ids.tolist() == [1, 3, -1] and top[2] == -np.inf
    np.testing.assert_allclose([ent, lse, top[0]], [np.log(2), 2 + np.log(2), -np.log(2)])
    lp, ent, lse, ids, _ = OT.stats_row(np.full(3, -np.inf), 1, 1)
    assert lp == lse == -np.inf and ent == 0 and ids.tolist() == [-1]


@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_stats_gradient_against_differences(scale):
    z = np.random.default_rng(1).standard_normal(9)
    f = lambda x: (lambda r: 0.8 * r[0] - 0.3 * r[1])(OT.stats_row(x, 4, 0, scale))  # noqa: E731
    np.testing.assert_allclose(OT.stats_grad_row(z, 4, 0.8, -0.3, scale), _diff(f, z), atol=1e-8)


def test_distill_closed_forms():
    z = np.log(np.array([0.1, 0.2, 0.3, 0.4]))
    assert OT.distill_row(z, [2, -1, 0, 1, 3], np.log([0.3, 9, 0.1, 0.2, 0.4]))[0] == pytest.approx(0, abs=1e-12)
    np.testing.assert_allclose(OT.distill_row(z, [3], [5.0])[0], -np.log(0.4))
    assert OT.distill_row(z, [-1, -1], [0.0, 1.0]) == (0.0, 0.0)
    np.testing.assert_allclose(OT.distill_row(z, [1, 1], [0.0, 0.0])[0], np.log(0.5) - np.log(0.2))


def test_distill_gradient_against_differences():
    rng = np.random.default_rng(2)
    z, ids, t = rng.standard_normal(7), np.array([5, -1, 2, 5]), np.array([0.3, 1.0, -np.inf, -0.4])
    np.testing.assert_allclose(OT.distill_grad_row(z, ids, t, 1.7, 0.8),
                               _diff(lambda x: 1.7 * OT.distill_row(x, ids, t, 0.8)[0], z), atol=1e-8)
