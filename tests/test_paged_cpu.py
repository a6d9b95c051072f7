"""Refusals of attention under a window and over pages and of norms with
rotation, which need no GPU: the C calls check sizes, strides and pointers before
any launch, the binding shapes, types, devices and layouts before any call."""
import ctypes
import math

import pytest
import torch

import chip_fusion_amd as cf

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x100000          # a device address that no refused call touches
F16 = torch.float16


def _t(*shape, dtype=F16):
    return torch.zeros(shape, dtype=dtype)


def _i(*v):
    return torch.tensor(v, dtype=torch.int32)


def _rows(p=P, ld=256, hs=64):
    return cf.Rows(p, ld, hs)


def _pages(p=P, ps=2048, ld=128, hs=64):
    return cf.Pages(p, ps, ld, hs)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(window=1 << 30, sinks=1 << 30), OK), (dict(dim=8), OK),
    (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(window=(1 << 30) + 1), INVALID), (dict(sinks=-1), INVALID),
    (dict(sinks=(1 << 30) + 1), INVALID), (dict(heads=0), INVALID), (dict(kv=3), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(dim=136), UNSUPPORTED), (dict(dim=12), UNSUPPORTED),
])
def test_create_window(kw, status):
    a = dict(dtype=0, heads=4, kv=2, dim=64, scale=1.0, window=5, sinks=2)
    a.update(kw)
    h = ctypes.c_void_p(5)
    st = cf.lib().b2b_attn_create_window(ctypes.byref(h), a["dtype"], a["heads"], a["kv"], a["dim"], a["scale"], a["window"],
                                         a["sinks"])
    assert st == status and bool(h.value) == (status == OK)
    if status == OK:
        assert cf.lib().b2b_attn_destroy(h) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(window=0, sinks=0), OK), (dict(page=7), OK), (dict(page=1 << 20), OK),
    (dict(page=0), INVALID), (dict(page=-4), INVALID), (dict(page=(1 << 20) + 1), INVALID), (dict(window=0), INVALID),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(heads=3), INVALID), (dict(dtype=3), UNSUPPORTED),
])
def test_create_paged(kw, status):
    a = dict(dtype=0, heads=4, kv=2, dim=64, page=16, scale=0.0, window=5, sinks=2)
    a.update(kw)
    h = ctypes.c_void_p(5)
    st = cf.lib().b2b_paged_attn_create(ctypes.byref(h), a["dtype"], a["heads"], a["kv"], a["dim"], a["page"], a["scale"],
                                        a["window"], a["sinks"])
    assert st == status and bool(h.value) == (status == OK)
    if status == OK:
        assert cf.lib().b2b_attn_destroy(h) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=-1), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 30), INVALID), (dict(width=-1), INVALID),
    (dict(width=1 << 26), INVALID),                                     # keys past 2^30
    (dict(pages=-1), INVALID), (dict(seqs=0, rows=0, cu=None), OK), (dict(rows=0), OK),     # nothing to do
    (dict(Q=_rows(None)), INVALID), (dict(Q=_rows(P + 8)), INVALID), (dict(Q=_rows(ld=252)), INVALID),
    (dict(K=_pages(None)), INVALID), (dict(K=_pages(P + 8)), INVALID), (dict(K=_pages(ps=2044)), INVALID),
    (dict(V=_pages(ld=12)), INVALID), (dict(V=_pages(hs=-64)), INVALID), (dict(V=_pages(ps=1 << 41)), INVALID),
    (dict(V=_pages(ps=1 << 40, hs=0), pages=1 << 20), INVALID),
    (dict(O=_rows()), INVALID), (dict(O=_rows(P * 2)), INVALID), (dict(O=_rows(P * 4, hs=0)), INVALID),
    (dict(table=None), INVALID), (dict(table_ld=255), INVALID), (dict(table_ld=-1), INVALID), (dict(lens=None), INVALID),
    (dict(cu=None), INVALID),                                           # 3 sequences, 4 rows
    (dict(lse=P + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=P + 8), INVALID), (dict(ws_bytes=15), INVALID),
    (dict(plan=None), INVALID),
])
def test_paged_run_refuses(kw, status):
    plan = cf.PagedAttention("f16", 4, 2, 64, 16)
    a = dict(plan=plan._h, seqs=3, rows=4, Q=_rows(), K=_pages(P * 2), V=_pages(P * 3), pages=100, table=P, width=256,
             table_ld=256, lens=P, cu=P, O=_rows(P * 4), lse=None, ws=P)
    n = ctypes.c_size_t()
    assert cf.lib().b2b_paged_attn_workspace(plan._h, 3, 4, 256, ctypes.byref(n)) == OK and n.value > 0
    a["ws_bytes"] = n.value
    a.update(kw)
    st = cf.lib().b2b_paged_attn_run(a["plan"], a["seqs"], a["rows"], a["Q"], a["K"], a["V"], a["pages"], a["table"], a["width"],
                                     a["table_ld"], a["lens"], a["cu"], a["O"], a["lse"], a["ws"], a["ws_bytes"], None)
    assert st == status


def test_plans_are_for_their_own_runs():
    """Plans of one kind are refused by the other kinds' calls, nothing launched."""
    L, n = cf.lib(), ctypes.c_size_t()
    paged, window = cf.PagedAttention("f16", 4, 2, 64, 16), cf.Attention("f16", 4, 2, 64, window=8)
    assert L.b2b_attn_workspace(paged._h, 1, 4, 100, ctypes.byref(n)) == INVALID
    assert L.b2b_attn_run(paged._h, 1, 4, 4, _rows(), _rows(P * 2), _rows(P * 3), _rows(P * 4), P, P, None, P, 1 << 30,
                          None) == INVALID
    assert L.b2b_paged_attn_workspace(window._h, 1, 4, 100, ctypes.byref(n)) == INVALID
    assert L.b2b_paged_attn_run(window._h, 3, 4, _rows(), _pages(P * 2), _pages(P * 3), 9, P, 2, 2, P, P, _rows(P * 4), None, P,
                                1 << 30, None) == INVALID
    for p in (paged, window):
        assert L.b2b_prefix_attn_run(p._h, 4, 10, 0, _rows(), _rows(P * 2), _rows(P * 3), _rows(None), 0, _rows(None), 0, None,
                                     _rows(P * 4), P, 1 << 30, None) == INVALID
    assert L.b2b_attn_workspace(window._h, 1, 1 << 30, 100, ctypes.byref(n)) == INVALID      # rows past 2^30 less one


def test_workspaces():
    """None where nothing can be cut; no more than 1024 slots of 128 rows."""
    n, L = ctypes.c_size_t(), cf.lib()
    plan = cf.PagedAttention("bf16", 32, 8, 128, 16)
    for seqs, rows, width, least in ((3, 3, 16, 0), (64, 64, 512, 1), (1, 1, 4096, 1), (300, 100000, 4096, 1)):
        assert L.b2b_paged_attn_workspace(plan._h, seqs, rows, width, ctypes.byref(n)) == OK
        assert (n.value > 0) == bool(least) and n.value <= 1024 * 128 * 129 * 4
    window = cf.Attention("bf16", 32, 8, 128, window=512, sinks=4)
    assert L.b2b_attn_workspace(window._h, 17, 8001, 8001, ctypes.byref(n)) == OK and n.value == 0      # tiles enough
    assert L.b2b_attn_workspace(window._h, 1, 40, 8001, ctypes.byref(n)) == OK and n.value > 0


@pytest.mark.parametrize("kw,match", [
    (dict(window=0), "window"), (dict(window=2.5), "window"), (dict(window=True), "window"), (dict(sinks=-1, window=4), "sinks"),
    (dict(sinks=4), "sinks"), (dict(window=4, causal=False), "window"), (dict(window=4, scale=0.0), "scale"),
])
def test_window_arguments(kw, match):
    with pytest.raises(ValueError, match=match):
        cf.Attention("f16", 4, 2, 64, **kw)


def test_binding_checks_paged():
    plan = cf.PagedAttention("f16", 4, 2, 64, 16)
    q, c, tab, lens = _t(3, 4, 64), _t(5, 16, 2, 64), _t(3, 6, dtype=torch.int32), _i(1, 2, 3)
    bad = [
        (dict(Q=_t(3, 3, 64)), "Q: shape"), (dict(K=c[:, :8]), "K: shape"), (dict(V=_t(4, 16, 2, 64)), "V: shape"),
        (dict(K=c.float()), "K: dtype"), (dict(K=[1]), "K: a torch"), (dict(K=_t(5, 16, 64, 2).transpose(2, 3)), "K: the last"),
        (dict(V=_t(5, 16, 2, 68)[..., :64]), "V: pages"), (dict(V=_t(5 * 2048 + 4)[4:].view(5, 16, 2, 64)), "V: pages"),
        (dict(table=tab.long()), "table"), (dict(table=tab[0]), "table"), (dict(table=_t(6, 3, dtype=torch.int32).t()), "table"),
        (dict(table=tab[:1].expand(3, 6)), "table"), (dict(lens=_i(1, 2)), "lens"), (dict(lens=lens.long()), "lens"),
        (dict(cu=_i(0, 3)), "cu: 4 values"), (dict(cu=_i(0, 1, 2, 3).float()), "cu"), (dict(Q=_t(4, 4, 64)), "cu: without"),
        (dict(O=_t(3, 4, 56)), "O: shape"), (dict(lse=_t(3, 4)), "lse"), (dict(), "device"),
    ]
    for kw, match in bad:
        a = dict(Q=q, K=c, V=c.clone(), table=tab, lens=lens)
        a.update(kw)
        with pytest.raises(ValueError, match=match):
            plan.run(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(rot=0, freqs=None), OK), (dict(axes=4, axes_of=[3] * 32), OK), (dict(flags=0, eps=-1.0), OK),
    (dict(heads=0), INVALID), (dict(kv=3), INVALID), (dict(rot=-8), INVALID), (dict(rot=72), INVALID),
    (dict(freqs=None), INVALID), (dict(freqs=[math.inf] * 32), INVALID), (dict(freqs=[math.nan] * 32), INVALID),
    (dict(axes=0), INVALID), (dict(axes=5), INVALID), (dict(axes=2, axes_of=[2] * 32), INVALID),
    (dict(axes_of=[-1] * 32), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=math.inf), INVALID), (dict(eps=math.nan), INVALID),
    (dict(flags=4), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(rot=60), UNSUPPORTED), (dict(dim=136), UNSUPPORTED),
    (dict(dim=68), UNSUPPORTED),
])
def test_create_rotary(kw, status):
    a = dict(dtype=0, heads=4, kv=2, dim=64, rot=64, freqs=[0.5] * 32, axes_of=None, axes=1, eps=1e-6, flags=1)
    a.update(kw)
    h = ctypes.c_void_p(5)
    f = None if a["freqs"] is None else (ctypes.c_double * 32)(*a["freqs"])
    x = None if a["axes_of"] is None else (ctypes.c_int * 32)(*a["axes_of"])
    st = cf.lib().b2b_rotary_create(ctypes.byref(h), a["dtype"], a["heads"], a["kv"], a["dim"], a["rot"], f, x, a["axes"],
                                    a["eps"], a["flags"])
    assert st == status and bool(h.value) == (status == OK)
    assert cf.lib().b2b_rotary_destroy(h if status == OK else None) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(rows=1 << 29), INVALID), (dict(rows=0), OK), (dict(plan=None), INVALID),
    (dict(Q=_rows(None)), INVALID), (dict(K=_rows(hs=4)), INVALID), (dict(Qo=_rows(P * 2)), INVALID),
    (dict(Ko=_rows(P)), INVALID), (dict(Qo=_rows(P * 4)), INVALID),          # over the keys, the queries, each other
    (dict(Qo=_rows(P, ld=512)), INVALID), (dict(Qo=_rows(P, hs=128, ld=512)), INVALID),      # in place at other strides
    (dict(Ko=_rows(P * 2, ld=64, hs=256)), INVALID), (dict(Qo=_rows(P * 3, hs=0)), INVALID),
    (dict(pos=None), INVALID), (dict(far=-4), INVALID), (dict(far=1 << 41), INVALID), (dict(qw=P + 8), INVALID),
    (dict(kw_=P + 2), INVALID),
])
def test_rotary_run_refuses(kw, status):
    plan = cf.NormRotary("f16", 4, 2, 64, sections=(16, 16))
    a = dict(plan=plan._h, rows=4, Q=_rows(), K=_rows(P * 2), Qo=_rows(P * 3), Ko=_rows(P * 4), pos=P, far=4, qw=None, kw_=None)
    a.update(kw)
    assert cf.lib().b2b_rotary_run(a["plan"], a["rows"], a["Q"], a["K"], a["Qo"], a["Ko"], a["pos"], a["far"], a["qw"], a["kw_"],
                                   None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=-1), INVALID), (dict(rows=-1), INVALID), (dict(rows=0), OK), (dict(seqs=0, cu=P), OK), (dict(cu=None), INVALID),
    (dict(pages=-1), INVALID), (dict(width=-1), INVALID), (dict(size=0), INVALID), (dict(size=(1 << 20) + 1), INVALID),
    (dict(V=_rows(None)), INVALID), (dict(Qo=_rows(P * 3)), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID),
    (dict(table_ld=3), INVALID), (dict(kc=_pages(None)), INVALID), (dict(kc=_pages(P * 6)), INVALID),       # values' pages
    (dict(kc=_pages(P)), INVALID), (dict(vc=_pages(P * 4)), INVALID), (dict(vc=_pages(P * 6, ps=0)), INVALID),
    (dict(kc=_pages(P * 5, ps=1024)), INVALID), (dict(kc=_pages(P * 5, ld=64)), INVALID),                   # rows overlap
    (dict(kc=_pages(P * 5, hs=56)), INVALID), (dict(kc=_pages(P * 5, ps=1024, ld=64, hs=512)), INVALID),
    (dict(far=-4), INVALID), (dict(qw=P + 8), INVALID), (dict(plan=None), INVALID),
])
def test_rotary_append_refuses(kw, status):
    plan = cf.NormRotary("f16", 4, 2, 64, sections=(16, 16))
    a = dict(plan=plan._h, seqs=3, rows=4, Q=_rows(), K=_rows(P * 2), V=_rows(P * 3), Qo=_rows(P * 4), kc=_pages(P * 5),
             vc=_pages(P * 6), pages=9, size=16, table=P, width=4, table_ld=4, lens=P, cu=P, pos=P, far=4, qw=None)
    a.update(kw)
    assert cf.lib().b2b_rotary_append(a["plan"], a["seqs"], a["rows"], a["Q"], a["K"], a["V"], a["Qo"], a["kc"], a["vc"],
                                      a["pages"], a["size"], a["table"], a["width"], a["table_ld"], a["lens"], a["cu"], a["pos"],
                                      a["far"], a["qw"], None, None) == status


@pytest.mark.parametrize("kw,match", [
    (dict(freqs=[1.0]), "freqs"), (dict(sections=(16, 15)), "sections"), (dict(sections=(40, -8)), "sections"),
    (dict(sections=(16, 16), axes_of=[0] * 32), "axes_of"), (dict(axes_of=[0] * 31), "axes_of"), (dict(base=0.0), "base"),
    (dict(base=-2.0), "base"), (dict(rotary_dim=-8), "rotary_dim"), (dict(rotary_dim=1.5), "rotary_dim"),
])
def test_rotary_arguments(kw, match):
    with pytest.raises(ValueError, match=match):
        cf.NormRotary("f16", 4, 2, 64, **kw)


def test_binding_checks_rotary():
    plan, plain = cf.NormRotary("f16", 4, 2, 64, sections=(16, 16)), cf.NormRotary("f16", 4, 2, 64, eps=None)
    q, k, pos, w = _t(3, 4, 64), _t(3, 2, 64), _t(2, 3, dtype=torch.int32), _t(64)
    bad = [
        (dict(Q=_t(3, 2, 64)), "Q: shape"), (dict(K=_t(2, 2, 64)), "K: shape"), (dict(positions=None), "positions"),
        (dict(positions=pos[0]), "positions"), (dict(positions=pos.long()), "positions"), (dict(positions=pos[:, :2]), "positions"),
        (dict(positions=_t(3, 2, dtype=torch.int32).t()), "positions"), (dict(q_weight=_t(63)), "q_weight"),
        (dict(k_weight=w.float()), "k_weight"), (dict(q_weight=_t(72)[4:68]), "q_weight"), (dict(Q_out=_t(3, 4, 56)), "Q_out"),
        (dict(K_out=_t(3, 3, 64)), "K_out"), (dict(), "device"),
    ]
    for kw, match in bad:
        a = dict(Q=q, K=k, positions=pos)
        a.update(kw)
        with pytest.raises(ValueError, match=match):
            plan.run(**a)
    with pytest.raises(ValueError, match="no norm"):
        plain.run(q, k, pos[0], q_weight=w)
    c, tab, lens = _t(5, 16, 2, 64), _t(3, 6, dtype=torch.int32), _i(1, 2, 3)
    bad = [
        (dict(V=_t(2, 2, 64)), "V: shape"), (dict(k_cache=_t(5, 16, 3, 64)), "k_cache: shape"),
        (dict(v_cache=_t(5, 8, 2, 64)), "v_cache: shape"), (dict(k_cache=_t(5, 0, 2, 64), v_cache=_t(5, 0, 2, 64)), "k_cache: a page"),
        (dict(table=tab[:2]), "lens"), (dict(cu=_i(0, 3)), "cu"), (dict(positions=pos[:1]), "positions"), (dict(), "device"),
    ]
    for kw, match in bad:
        a = dict(Q=q, K=k, V=k.clone(), k_cache=c, v_cache=c.clone(), table=tab, lens=lens)
        a.update(kw)
        with pytest.raises(ValueError, match=match):
            plan.append(**a)


def test_closed_plans():
    for plan in (cf.PagedAttention("f16", 4, 2, 64, 16), cf.NormRotary("f16", 4, 2, 64), cf.Attention("f16", 4, 2, 64, window=3)):
        plan.close()
        plan.close()
        assert plan._h is None
