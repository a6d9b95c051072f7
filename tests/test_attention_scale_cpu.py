"""Scales of the attention plans that float32 does not hold."""
import ctypes

import pytest

import chip_fusion_amd as cf

PLANS = [lambda s: cf.Attention("f16", 2, 2, 64, scale=s), lambda s: cf.PrefixAttention("bf16", 2, 2, 64, scale=s),
         lambda s: cf.LinearAttention("f16", 2, 2, 64, scale=s)]


@pytest.mark.parametrize("make", PLANS)
def test_a_scale_that_rounds_to_0_is_refused(make):
    """0 asks the library for its default, which is another scale."""
    for scale in (1e-46, 1e-300):
        with pytest.raises(ValueError, match="scale"):
            make(scale)
    for scale in (1e-45, 1e-38, 1e38):        # float32's smallest, a subnormal one, a large one
        make(scale).close()
    for scale in (1e39, float("inf")):
        with pytest.raises(cf.B2BError, match="invalid"):
            make(scale)
