"""The two forms of the dQ pass (two blocks per SM for many short lists, one
otherwise): each against the float64 oracle, with the bounds of
test_gpu_window.py, and with the same bits as the other.  The form follows the
number of tile pairs that the descriptor bounds, so a loose bound takes the
second form."""
import numpy as np
import pytest

from oracle import window as OW
from sft_trie_build_gb300 import stp
from test_gpu_window import Run, _check, _forest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (4, 2)])
@pytest.mark.parametrize("window", [20, 2 ** 31 - 1])
def test_many_short_rows(hq, hkv, window):
    plan = _forest(21, 256, n_roots=60, max_depth=2, len_hi=70)
    assert plan.n_rows >= 24          # enough blocks for two per SM to be taken
    _check(Run(plan.subtree_end, plan.position_ids, hq, hkv, 128, stp.STP_BF16, window, 2, seed=hq), OW.mask(plan, window, 2))


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2)])
def test_same_bits_in_both_forms(hq, hkv):
    plan = _forest(22, 2048, n_roots=80, max_depth=3, len_lo=10, len_hi=200)
    se, pos = plan.subtree_end[:8], plan.position_ids[:8]
    assert len(se) == 8
    a, b = (Run(se, pos, hq, hkv, 128, stp.STP_BF16, 100, 0, seed=3) for _ in range(2))
    tiles = 8 * 16
    assert 25 * a.pairs <= tiles * tiles < 25 * 8 * 16 * 17 // 2
    b.desc = stp.Desc(8, 2048, hq, hkv, 128, stp.STP_BF16, 0.0, 0, 0)     # every pair below the diagonal
    b.buf = stp.Buffers(b.desc)
    a.step()
    b.step()
    x, y = a.outputs(), b.outputs()
    for n in x:
        assert np.array_equal(x[n], y[n]), n
