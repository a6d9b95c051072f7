"""Outputs that share elements with other operands: the rule that tells them from
outputs between others' rows, under sanitizers against sets of elements, and the
calls that refuse them before any launch."""
import ctypes
import os

import pytest

import chip_fusion_amd as cf
from test_paged_cpu import INVALID, P, _pages, _rows
from test_sanitizers import CSRC, HERE, _build_and_run


def test_overlaps_against_sets_of_elements(tmp_path):
    out = _build_and_run(tmp_path, "g++", [os.path.join(HERE, "extent_driver.cpp")], ["-std=c++17", "-I", CSRC])
    assert ", 0 wrong" in out


# Q (4 heads) and K (2 heads) of 64, rows of 512 elements (1024 bytes), at P and P + 512
@pytest.mark.parametrize("kw", [
    dict(Qo=_rows(P + 1024, 512)),                  # a row further than the queries
    dict(Qo=_rows(P - 1024, 512)), dict(Qo=_rows(P + 3 * 1024, 512)),
    dict(Qo=_rows(P + 128, 512)),                   # a head further, over keys as well
    dict(Qo=_rows(P * 2 + 640, 512), Ko=_rows(P * 2 + 512, 512)),       # over each other
    dict(Qo=_rows(P + 2048 + 768, 256)),            # dense, over keys of one row
    dict(Ko=_rows(P + 512 + 1024, 512)),            # a row further than the keys
    dict(Ko=_rows(P + 256, 512)), dict(Ko=_rows(P + 64, 512)), dict(Ko=_rows(P + 16, 128)),
    dict(Qo=_rows(P * 2, 64, 320), Ko=_rows(P * 2 + 496, 128)),         # heads first, keys in its gaps and on its heads
])
def test_rotations_refuse_outputs_over_operands(kw):
    plan = cf.NormRotary("f16", 4, 2, 64)
    a = dict(Q=_rows(P, 512), K=_rows(P + 512, 512), Qo=_rows(P * 3), Ko=_rows(P * 4))
    a.update(kw)
    assert cf.lib().b2b_rotary_run(plan._h, 4, a["Q"], a["K"], a["Qo"], a["Ko"], P * 6, 4, None, None, None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(Qo=_rows(P + 1024, 512)), dict(Qo=_rows(P + 512, 512)), dict(Qo=_rows(P + 768, 512)),      # queries, keys, values
    dict(Qo=_rows(P * 5 + 4096)), dict(Qo=_rows(P * 6 + 9 * 4096 - 128)),                           # pages
    dict(kc=_pages(P + 1024)), dict(vc=_pages(P - 4096 * 8)), dict(kc=_pages(P + 3 * 1024 + 896)),
    dict(kc=_pages(P * 5, 4096), vc=_pages(P * 5 + 2048, 4096)),                                    # half a page further
    dict(vc=_pages(P * 5 + 8 * 4096)), dict(vc=_pages(P * 5 + 4096 * 4 + 128)),
    dict(kc=_pages(P * 5, 8192, 256, 128), vc=_pages(P * 5 + 128, 8192, 256, 64)),
])
def test_appends_refuse_pages_over_operands(kw):
    """Pages of 16 rows of 2 heads of 64: 2048 elements, 4096 bytes."""
    plan = cf.NormRotary("f16", 4, 2, 64)
    a = dict(Q=_rows(P, 512), K=_rows(P + 512, 512), V=_rows(P + 768, 512), Qo=_rows(P * 4), kc=_pages(P * 5), vc=_pages(P * 6))
    a.update(kw)
    assert cf.lib().b2b_rotary_append(plan._h, 3, 4, a["Q"], a["K"], a["V"], a["Qo"], a["kc"], a["vc"], 9, 16, P * 8, 4, 4, P * 8,
                                      P * 8, None, 0, None, None, None) == INVALID
