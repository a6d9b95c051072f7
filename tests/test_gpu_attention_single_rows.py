"""Calls of one row, whose row stride nothing steps by: any stride of any tensor
gives what a dense call gives, and nothing else is written."""
import math

import pytest
import torch

import chip_fusion_amd as cf

pytestmark = pytest.mark.gpu

H, D = 3, 64


def _flush(msg):
    print(f"\n[case] {msg}", flush=True)


def _randn(seed, shape, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _strided(x, ld):
    """x, in room of its own, as a row whose next would be ld elements on."""
    room = torch.empty((x.numel(),), dtype=x.dtype, device="cuda").copy_(x.reshape(-1))
    return room.as_strided((1, H, D), (ld, D, 1))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("ld", [1 << 27, (1 << 27) + 8, 1 << 31, 1 << 40, 1 << 24, H * D + 8])
def test_any_row_stride(dtype, ld):
    """(2^27 elements and 16 rows are 2^32 bytes.)"""
    name = "f16" if dtype is torch.float16 else "bf16"
    _flush(f"one row {name} {ld}")
    q, k, v = (_randn(i, (1, H, D), dtype) for i in (1, 2, 3))
    s0, g = _randn(4, (1, H, D, D), torch.float32), torch.full((H,), -0.3, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    far = tuple(_strided(x, ld) for x in (q, k, v))
    room = torch.full((H * D + 4096,), 7.0, dtype=dtype, device="cuda")
    O = room.as_strided((1, H, D), (ld, D, 1))

    def same(want):
        torch.cuda.synchronize()
        assert torch.equal(O, want) and bool((room[H * D:] == 7.0).all())
        room.fill_(7.0)

    lin, att = cf.LinearAttention(name, H, H, D), cf.Attention(name, H, H, D)
    for stream in (None, torch.cuda.current_stream()):        # compiled and in Python
        (want, ws), (_, s) = lin.run(q, k, v, g, cu, state=s0), lin.run(*far, g, cu, state=s0, O=O, stream=stream)
        same(want)
        assert torch.equal(s, ws)
        (want, ws), (_, s) = lin.step(q, k, v, g, s0), lin.step(*far, g, s0, O=O, stream=stream)
        same(want)
        assert torch.equal(s, ws)
        want = att.run(q, k, v, cu)
        att.run(*far, cu, O=O, stream=stream)
        same(want)


@pytest.mark.parametrize("ld", [0, -64, 8])
def test_strides_below_a_row(ld):
    """Through the C call, which takes them where there is one row."""
    _flush(f"one row, stride {ld}")
    q, k, v = (_randn(i, (1, H, D), torch.float16) for i in (1, 2, 3))
    g, cu = torch.full((H,), -0.3, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    plan = cf.LinearAttention("f16", H, H, D)
    want, ws = plan.run(q, k, v, g, cu)
    room, after = torch.full((H * D + 4096,), 7.0, dtype=torch.float16, device="cuda"), torch.full_like(ws, math.nan)
    rows = lambda t: cf.Rows(t.data_ptr(), ld, D)
    assert cf.lib().b2b_linear_attn_run(plan._h, 1, 1, rows(q), rows(k), rows(v), rows(room), g.data_ptr(), cu.data_ptr(),
                                        None, after.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(room[:H * D], want.reshape(-1)) and bool((room[H * D:] == 7.0).all()) and torch.equal(after, ws)
