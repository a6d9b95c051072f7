"""Outputs that lie between their operands' rows, as slices of one tensor do, are
taken: queries turned in place in a fused projection, keys and values side by side
in every order of a cache's dimensions."""
import pytest
import torch

import chip_fusion_amd as cf
from test_gpu_norm_rotary import _flush, _int, _randn

pytestmark = pytest.mark.gpu


def _split(fused, H, Hkv):
    return fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:]


@pytest.mark.parametrize("T,H,Hkv", [(1, 4, 2), (1, 1, 1), (7, 4, 1), (300, 8, 2)])
@pytest.mark.parametrize("heads_first", [False, True])
def test_in_place_in_a_fused_projection(T, H, Hkv, heads_first):
    _flush(f"in place, {T} rows of {H} + {Hkv} heads, heads first {heads_first}")
    D, n = 64, H + 2 * Hkv
    fused = _randn(1, (n, T, D) if heads_first else (T, n, D), torch.bfloat16)
    if heads_first:
        fused = fused.transpose(0, 1)
    q, k, v = _split(fused, H, Hkv)
    kept, pos, plan = v.clone(), _int(range(T)), cf.NormRotary("bf16", H, Hkv, D)
    want = plan.run(q.contiguous(), k.contiguous(), pos)
    got = plan.run(q, k, pos, Q_out=q, K_out=k)
    torch.cuda.synchronize()
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)


CACHES = [                  # shape in memory, and the order that makes it [2, pages, size, heads, dim]
    ((9, 2, 16, 2, 64), (1, 0, 2, 3, 4)), ((9, 16, 2, 2, 64), (2, 0, 1, 3, 4)), ((9, 16, 2, 2, 64), (3, 0, 1, 2, 4)),
    ((2, 9, 2, 16, 64), (0, 1, 3, 2, 4)), ((9, 2, 2, 16, 64), (1, 0, 3, 2, 4)), ((16, 2, 9, 2, 64), (1, 2, 0, 3, 4)),
]


@pytest.mark.parametrize("case", range(len(CACHES)))
def test_append_into_keys_and_values_side_by_side(case):
    _flush(f"append, cache {CACHES[case]}")
    H, Hkv, D, dt = 4, 2, 64, torch.float16
    fused = _randn(2, (5, H + 2 * Hkv, D), dt)
    q, k, v = _split(fused, H, Hkv)
    table, lens, cu = _int([[3, 8, -1], [0, 5, 2]]), _int([17, 40]), _int([0, 2, 5])
    plan = cf.NormRotary("f16", H, Hkv, D)
    plain = [torch.full((9, 16, Hkv, D), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    want = plan.append(q.contiguous(), k.contiguous(), v.contiguous(), *plain, table, lens, cu)
    shape, order = CACHES[case]
    both = torch.full(shape, 7.0, dtype=dt, device="cuda").permute(order)
    plan.append(q, k, v, both[0], both[1], table, lens, cu, Q_out=q)
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(both[0], plain[0]) and torch.equal(both[1], plain[1])
    attn = cf.PagedAttention("f16", H, Hkv, D, 16)
    a, b = attn.run(want, *plain, table, lens, cu), attn.run(q, both[0], both[1], table, lens, cu, O=q.new_empty(q.shape))
    torch.cuda.synchronize()
    assert torch.equal(a, b)
