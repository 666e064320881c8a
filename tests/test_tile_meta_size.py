"""The size of tile_meta: what tree attention without a window needs, and at
most 12 bytes per token and 4 KiB more for the windowed calls, which share the
arrays of [R, NT, NT] entries."""
import pytest

from sft_trie_build_gb300 import stp


@pytest.mark.parametrize("rows,row_len", [(1, 128), (3, 512), (1, 16384), (16, 4096), (1, 131072), (1000, 256)])
def test_windows_cost_plain_attention_little(stp_lib, rows, row_len):
    nt = row_len // 128
    # classes, two lists, ranks, pair indices; four counts or extremes a tile, an offset; a base a row
    plain = rows * nt * nt * (1 + 4 * 4) + rows * nt * 5 * 4 + rows * 4 + 12 * 256
    meta, _, _ = stp.stp_workspace_size(stp.Desc(rows, row_len, 1, 1, 128))
    assert meta <= plain + 12 * rows * row_len + 4096
