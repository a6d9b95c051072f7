"""Norms of queries and keys whose weights and elements are of opposite extremes."""
import pytest
import torch

import chip_fusion_amd as cf
import paged_ref as R
from test_gpu_norm_rotary import _flush, _int, _randn

pytestmark = pytest.mark.gpu


# input's size, weights' sizes (powers of two)
@pytest.mark.parametrize("x,ws", [(58, (100, 0)), (-45, (-110, 0)), (0, (120, -120)), (50, (-120, 60)), (-48, (61, -61)), (40, (90, 90)), (-45, (-110, -110))])
@pytest.mark.parametrize("inter", [False, True])
def test_weights_of_any_size(x, ws, inter):
    """The norm's factor and the weight may be of opposite extremes: their product
    with the element leaves float32's range, the result does not."""
    _flush(f"weights of 2^{ws}, heads of 2^{x}, interleaved {inter}")
    H, D, T, dt = 2, 64, 5, torch.bfloat16
    q, k = (_randn(i, (T, H, D), dt) * 2.0 ** x for i in (1, 2))
    w = [_randn(3 + i, (D,), dt, 0.2, 1.0) for i in range(2)]
    size = torch.where(torch.arange(D) % 3 == 0, ws[0], ws[1]).double()
    w = [(y.cpu().double() * 2.0 ** size).to(dt).cuda() for y in w]
    pos = _int([0, 1, 7, 1000, 123456])
    got = cf.NormRotary("bf16", H, H, D, interleaved=inter, eps=0.0).run(q, k, pos, *w)
    torch.cuda.synchronize()
    for a, b, y in ((q, w[0], got[0]), (k, w[1], got[1])):
        want, bound = R.norm_rotary(a, b, pos[None], D, R.default_freqs(D), None, inter, 0.0)
        R.check(y, want, bound + 2.0 ** -134)          # (bf16's subnormal steps: 2^-133)
