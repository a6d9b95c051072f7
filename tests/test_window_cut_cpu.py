"""Which calls under a window have their keys cut: those of which one row tile may
have many more keys than the others, whatever the number of rows."""
import ctypes

import pytest

import chip_fusion_amd as cf


def _bytes(call, plan, *sizes):
    n = ctypes.c_size_t()
    assert getattr(cf.lib(), call)(plan._h, *sizes, ctypes.byref(n)) == 0
    return n.value


# window, sequences, rows, keys that the table holds, cut
@pytest.mark.parametrize("window,seqs,rows,keys,cut", [
    (32768, 4, 2048, 16384, True),              # as wide as the contexts: as without a window
    (1 << 30, 61, 2464, 100064, True),          # one chunk behind many keys among short prompts
    (4096, 61, 2464, 16384, True),
    (512, 4, 2048, 16384, False),               # row tiles enough, none with many more keys
    (512, 4, 2048, 1 << 26, False),
    (4096, 1, 32768, 32768, False),             # 8192 row tiles beside which 134 key tiles are little
    (1 << 30, 1, 32768, 1 << 20, True),
    (64, 4, 100, 16384, False),                 # nothing to cut
    (1000, 1, 40, 16384, True),                 # few rows
])
def test_pages(window, seqs, rows, keys, cut):
    plan = cf.PagedAttention("bf16", 32, 8, 128, 64, window=window, sinks=4)
    got = _bytes("b2b_paged_attn_workspace", plan, seqs, rows, -(-keys // 64))
    assert (got > 0) == cut
    if cut and window >= keys:                  # no more than without a window
        assert got <= _bytes("b2b_paged_attn_workspace", cf.PagedAttention("bf16", 32, 8, 128, 64), seqs, rows, -(-keys // 64))


@pytest.mark.parametrize("window,rows,keys,cut", [
    (4096, 32768, 32768, False), (512, 8001, 8001, False), (1 << 30, 8001, 8001, False),        # prompts from their beginning
    (1 << 30, 8001, 100000, True), (4096, 2464, 20000, True), (512, 2464, 100000, False),       # pieces behind earlier keys
])
def test_side_by_side(window, rows, keys, cut):
    plan = cf.Attention("bf16", 32, 8, 128, window=window, sinks=4)
    assert (_bytes("b2b_attn_workspace", plan, 17, rows, keys) > 0) == cut
