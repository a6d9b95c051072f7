"""Numbers of sequences, places and pages past the library's 32 bits are refused, not
taken modulo 2^32 (tensors without memory)."""
import pytest
import torch

import chip_fusion_amd as cf

N = 2 ** 32 + 1


def _h(*shape):
    return torch.empty((1,), dtype=torch.float16, device="meta").expand(shape) if N in shape else \
        torch.empty(shape, dtype=torch.float16, device="meta")


def _i(*shape):
    return torch.empty(shape, dtype=torch.int32, device="meta")


@pytest.mark.parametrize("kw,match", [
    (dict(table=_i(1, N)), "table"), (dict(table=_i(N, 1), lens=_i(N), cu=_i(N + 1)), "table"),
    (dict(k_cache=_h(N, 16, 2, 64), v_cache=_h(N, 16, 2, 64)), "fewer than 2.31 pages"),
])
def test_counts(kw, match):
    a = dict(Q=_h(1, 4, 64), k_cache=_h(9, 16, 2, 64), v_cache=_h(9, 16, 2, 64), table=_i(1, 3), lens=_i(1), cu=None)
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        cf.PagedAttention("f16", 4, 2, 64, 16).run(*a.values())
    Q, kc, vc, table, lens, cu = a.values()
    with pytest.raises(ValueError, match=match):
        cf.NormRotary("f16", 4, 2, 64).append(Q, _h(1, 2, 64), _h(1, 2, 64), kc, vc, table, lens, cu)
