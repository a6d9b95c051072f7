"""Many rows under a window whose keys are cut all the same: a chunk and single
tokens behind long contexts among prompts that begin."""
import pytest
import torch

import chip_fusion_amd as cf
import paged_ref as R
from test_gpu_norm_rotary import DT, _flush, _int, _pool, _randn
from test_gpu_paged_attention import _fill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,size", [("bf16", 64, 16), ("f16", 96, 24)])
@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), (2100, 40)])
def test_a_far_chunk_among_prompts(dtype, D, size, window, sinks):
    _flush(f"a far chunk, {dtype} {D}, window {window}")
    H, Hkv = 32, 8
    lq = [34] * 30 + [70, 1, 1] + [33] * 31
    lk = [n if n > 1 and n != 70 else n + 2900 for n in lq]
    kc, vc, table = _pool(1, lk, size, Hkv, D, DT[dtype])
    k, v = _fill(kc, table, lk, 2), _fill(vc, table, lk, 3)
    q = _randn(1, (sum(lq), H, D), DT[dtype], 1.5)
    want, want_lse, b, bl = R.attend(q, k, v, lq, lk, window, sinks)
    cu, n = _int(R.starts(lq)), _int(lk)
    pages = cf.PagedAttention(dtype, H, Hkv, D, size, window=window, sinks=sinks)
    got, lse = pages.run(q, kc, vc, table, n, cu, lse=True)
    rows, row_lse = cf.Attention(dtype, H, Hkv, D, window=window, sinks=sinks).run(q, k, v, cu, _int(R.starts(lk)), lse=True)
    again = pages.run(q, kc, vc, table, n, cu)
    torch.cuda.synchronize()
    for o, l, what in ((got, lse, "pages"), (rows, row_lse, "side by side")):
        R.check(o, want, b, what)
        R.check(l, want_lse, bl, what + " LSE")
    assert torch.equal(again, got)
