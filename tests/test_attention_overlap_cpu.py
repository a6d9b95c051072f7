"""Attention over pages and under a window refuses an output that shares elements
with an input, before any launch."""
import pytest

import chip_fusion_amd as cf
from test_paged_cpu import INVALID, P, _pages, _rows

# Q of 4 rows of 4 heads of 64, 1024 bytes a row; keys of 2 heads
OVER_QUERIES = [_rows(P + 1024, 512), _rows(P + 128, 512), _rows(P - 2048, 512), _rows(P + 3 * 1024 + 384), _rows(P + 256, 64, 512)]


@pytest.mark.parametrize("O", OVER_QUERIES + [
    _rows(P * 2 + 4096), _rows(P * 2 - 1024), _rows(P * 3 + 99 * 4096 + 3968), _rows(P * 3 + 5 * 4096 + 1024, 128, 512)])
def test_paged(O):
    plan = cf.PagedAttention("f16", 4, 2, 64, 16)
    st = cf.lib().b2b_paged_attn_run(plan._h, 4, 4, _rows(P, 512), _pages(P * 2), _pages(P * 3), 100, P * 8, 4, 4, P * 8, P * 8, O,
                                     None, None, 0, None)
    assert st == INVALID


@pytest.mark.parametrize("O", OVER_QUERIES + [_rows(P * 2 + 512), _rows(P * 3 - 512), _rows(P * 3 + 99 * 256 + 128)])
def test_window(O):
    plan = cf.Attention("f16", 4, 2, 64, window=8)
    st = cf.lib().b2b_attn_run(plan._h, 1, 4, 100, _rows(P, 512), _rows(P * 2, 128), _rows(P * 3, 128), O, P * 8, P * 8, None,
                               None, 0, None)
    assert st == INVALID
