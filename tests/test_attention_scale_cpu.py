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


@pytest.mark.parametrize("scale,status", [(2.3e38, 0), (2.4e38, 1), (3.4e38, 1)])
def test_a_scale_whose_base_2_form_is_infinite_is_refused(scale, status):
    """(Scores of 0 would be 0 times infinity.)"""
    h = ctypes.c_void_p()
    assert cf.lib().b2b_attn_create(ctypes.byref(h), 0, 2, 2, 64, scale, 0) == status
    assert bool(h.value) == (status == 0)
    cf.lib().b2b_attn_destroy(h)
