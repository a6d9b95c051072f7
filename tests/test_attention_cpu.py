"""The attention operators' refusals, which need no GPU: the C calls check
sizes, strides and pointers before any launch, the binding shapes, types,
devices and layouts before any call."""
import ctypes
import os
import re

import pytest
import torch

import chip_fusion_amd as cf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x100000          # a device address that no refused call touches


def test_exports_every_declared_symbol():
    txt = open(os.path.join(ROOT, "include", "b2b_attn.h")).read()
    names = set(re.findall(r"\b(b2b_[a-z0-9_]+)\s*\(", txt))
    assert names == set(cf.ATTN_EXPORTS)
    for n in names:
        assert hasattr(cf.lib(), n)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(dtype=1, heads=8, kv=1, dim=8), OK), (dict(scale=0.0), OK),
    (dict(heads=0), INVALID), (dict(kv=0), INVALID), (dict(kv=3), INVALID), (dict(dim=0), INVALID),
    (dict(flags=2), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(dim=132), UNSUPPORTED), (dict(dim=136), UNSUPPORTED),
    (dict(dim=12), UNSUPPORTED),
])
def test_create(kw, status):
    a = dict(dtype=0, heads=4, kv=2, dim=64, scale=1.0, flags=0)
    a.update(kw)
    h = ctypes.c_void_p(5)
    st = cf.lib().b2b_attn_create(ctypes.byref(h), a["dtype"], a["heads"], a["kv"], a["dim"], a["scale"], a["flags"])
    assert st == status and bool(h.value) == (status == OK)
    if status == OK:
        assert cf.lib().b2b_attn_destroy(h) == OK
    assert cf.lib().b2b_attn_destroy(None) == OK


def _rows(p=P, ld=256, hs=64):
    return cf.Rows(p, ld, hs)


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=-1), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(keys=1 << 31), INVALID),
    (dict(rows=1 << 30), INVALID),                          # rows x heads past 2^31
    (dict(seqs=0), OK), (dict(rows=0), OK),                 # nothing to do
    (dict(Q=_rows(None)), INVALID), (dict(Q=_rows(P + 8)), INVALID), (dict(Q=_rows(ld=252)), INVALID),
    (dict(Q=_rows(ld=56)), INVALID), (dict(K=_rows(hs=4)), INVALID), (dict(K=_rows(hs=-64)), INVALID),
    (dict(V=_rows(ld=(1 << 23) + 8)), INVALID), (dict(V=_rows(None)), INVALID),
    (dict(O=_rows()), INVALID),                             # O at Q's address
    (dict(O=_rows(P * 4, hs=0)), INVALID), (dict(O=_rows(P * 4, hs=56)), INVALID),      # heads of O overlap
    (dict(O=_rows(P * 4, ld=192)), INVALID), (dict(O=_rows(P * 4, ld=64, hs=192)), INVALID),
    (dict(Q=_rows(hs=1 << 41)), INVALID),
    (dict(cu_q=None), INVALID), (dict(cu_k=None), INVALID), (dict(lse=P + 2), INVALID),
    (dict(ws=None), INVALID), (dict(ws=P + 8), INVALID), (dict(ws_bytes=15), INVALID),
    (dict(plan=None), INVALID),
])
def test_run_refuses(kw, status):
    plan = cf.Attention("f16", 4, 2, 64)
    a = dict(plan=plan._h, seqs=1, rows=4, keys=4096, Q=_rows(), K=_rows(P * 2), V=_rows(P * 3), O=_rows(P * 4), cu_q=P,
             cu_k=P, lse=None, ws=P, ws_bytes=0)
    n = ctypes.c_size_t()
    assert cf.lib().b2b_attn_workspace(plan._h, 1, 4, 4096, ctypes.byref(n)) == OK
    assert n.value > 0                                      # few rows, many keys: partial results
    a["ws_bytes"] = n.value
    a.update(kw)
    st = cf.lib().b2b_attn_run(a["plan"], a["seqs"], a["rows"], a["keys"], a["Q"], a["K"], a["V"], a["O"], a["cu_q"],
                               a["cu_k"], a["lse"], a["ws"], a["ws_bytes"], None)
    assert st == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(prefix=-1), INVALID), (dict(own=-1), INVALID), (dict(own=1 << 31), INVALID),
    (dict(batch=0), OK), (dict(Q=_rows(None)), INVALID), (dict(Kp=_rows(None)), INVALID), (dict(V=_rows(ld=8)), INVALID),
    (dict(ks=12), INVALID), (dict(vs=-8), INVALID), (dict(lens=None), INVALID), (dict(O=_rows()), INVALID),
    (dict(O=_rows(P * 6, hs=0)), INVALID), (dict(ks=1 << 41), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=16), INVALID), (dict(causal=True), INVALID),
])
def test_prefix_run_refuses(kw, status):
    a = dict(batch=4, prefix=100, own=10, Q=_rows(), Kp=_rows(P * 2), Vp=_rows(P * 3), K=_rows(P * 4), ks=640, V=_rows(P * 5),
             vs=640, lens=P, O=_rows(P * 6), ws=P, causal=False, ws_bytes=1 << 30)
    a.update(kw)
    plan = cf.Attention("f16", 4, 2, 64, causal=a["causal"])
    st = cf.lib().b2b_prefix_attn_run(plan._h, a["batch"], a["prefix"], a["own"], a["Q"], a["Kp"], a["Vp"], a["K"],
                                      a["ks"], a["V"], a["vs"], a["lens"], a["O"], a["ws"], a["ws_bytes"], None)
    assert st == status


def _t(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


def _cu(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_binding_checks_attention():
    plan = cf.Attention("f16", 4, 2, 64)
    q, k, v, cu = _t(10, 4, 64), _t(10, 2, 64), _t(10, 2, 64), _cu(0, 10)
    bad = [
        (dict(Q=q.float()), "Q: dtype"), (dict(Q=_t(10, 3, 64)), "Q: shape"), (dict(K=_t(10, 2, 32)), "K: shape"),
        (dict(V=_t(9, 2, 64)), "V: shape"), (dict(Q=[1]), "Q: a torch tensor"),
        (dict(Q=_t(10, 4, 128)[:, :, ::2]), "Q: the last dimension"),
        (dict(K=_t(10 * 128 + 4)[4:].view(10, 2, 64)), "K: rows and heads must start"),
        (dict(K=_t(10, 2 * 64 + 4)[:, :128].view(10, 2, 64)), "K: rows and heads must start"),
        (dict(V=_t(1, 2, 64).expand(10, 2, 64)), "V: rows overlap"),
        (dict(cu_q=cu.long()), "cu_q"), (dict(cu_q=_cu(0, 4, 10), cu_k=cu), "cu_k: 3 values"), (dict(cu_q=_cu()), "cu_q"),
        (dict(O=_t(10, 4, 63)), "O: shape"), (dict(lse=_t(10, 4)), "lse"), (dict(lse=_t(10, 3, dtype=torch.float32)), "lse"),
        (dict(), "device"),                       # everything fits, but in host memory
    ]
    for kw, match in bad:
        a = dict(Q=q, K=k, V=v, cu_q=cu)
        a.update(kw)
        with pytest.raises(ValueError, match=match):
            plan.run(**a)
    with pytest.raises(ValueError, match="scale"):
        cf.Attention("f16", 4, 2, 64, scale=-1.0)
    with pytest.raises(cf.B2BError, match="not supported"):
        cf.Attention("f64", 4, 2, 64)
    plan.close()


def test_binding_checks_prefix():
    plan = cf.PrefixAttention("bf16", 4, 2, 64)
    T = torch.bfloat16
    q, kp, k = _t(3, 4, 64, dtype=T), _t(7, 2, 64, dtype=T), _t(3, 5, 2, 64, dtype=T)
    lens = _cu(1, 2, 3)
    for kw, match in [
        (dict(Kp=_t(7, 2, 64)), "Kp: dtype"), (dict(Vp=kp[:6]), "Vp: shape"), (dict(K=k[:2]), "K: shape"),
        (dict(V=k[:, :4]), "V: shape"), (dict(lens=_cu(1, 2)), "lens"), (dict(lens=lens.long()), "lens"),
        (dict(K=_t(3 * 644, dtype=T).as_strided((3, 5, 2, 64), (644, 128, 64, 1))), "K: requests must start"),
        (dict(), "device"),
    ]:
        a = dict(Q=q, Kp=kp, Vp=kp, K=k, V=k, lens=lens)
        a.update(kw)
        with pytest.raises(ValueError, match=match):
            plan.run(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(dtype=1, dim=128), OK), (dict(heads=0), INVALID), (dict(kv=3), INVALID), (dict(dim=-1), INVALID),
    (dict(scale=-2.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(dim=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
])
def test_linear_create(kw, status):
    a = dict(dtype=0, heads=4, kv=2, dim=64, scale=1.0)
    a.update(kw)
    h = ctypes.c_void_p(5)
    st = cf.lib().b2b_linear_attn_create(ctypes.byref(h), a["dtype"], a["heads"], a["kv"], a["dim"], a["scale"])
    assert st == status and bool(h.value) == (status == OK)
    if status == OK:
        assert cf.lib().b2b_linear_attn_destroy(h) == OK
    assert cf.lib().b2b_linear_attn_destroy(None) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=-1), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 30), INVALID), (dict(seqs=0), OK),
    (dict(Q=_rows(None)), INVALID), (dict(K=_rows(ld=100)), INVALID), (dict(V=_rows(P + 4)), INVALID), (dict(O=_rows()), INVALID),
    (dict(O=_rows(P * 4, ld=128)), INVALID),
    (dict(g=None), INVALID), (dict(cu=None), INVALID), (dict(s0=P + 4), INVALID), (dict(s1=P + 8), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=64), INVALID), (dict(ws=P + 8), INVALID), (dict(plan=None), INVALID),
])
def test_linear_run_refuses(kw, status):
    plan = cf.LinearAttention("f16", 4, 2, 64)
    a = dict(plan=plan._h, seqs=1, rows=5000, Q=_rows(), K=_rows(P * 2), V=_rows(P * 3), O=_rows(P * 4), g=P, cu=P, s0=P,
             s1=P, ws=P)
    n = ctypes.c_size_t()
    assert cf.lib().b2b_linear_attn_workspace(plan._h, 1, 5000, ctypes.byref(n)) == OK and n.value > 0
    a["ws_bytes"] = n.value
    a.update(kw)
    st = cf.lib().b2b_linear_attn_run(a["plan"], a["seqs"], a["rows"], a["Q"], a["K"], a["V"], a["O"], a["g"], a["cu"],
                                      a["s0"], a["s1"], a["ws"], a["ws_bytes"], None)
    assert st == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(batch=0), OK), (dict(Q=_rows(None)), INVALID), (dict(O=_rows()), INVALID),
    (dict(s0=None), INVALID), (dict(s1=None), INVALID), (dict(s0=P + 8), INVALID), (dict(g=None), INVALID),
])
def test_linear_step_refuses(kw, status):
    plan = cf.LinearAttention("f16", 4, 2, 64)
    a = dict(batch=3, Q=_rows(), K=_rows(P * 2), V=_rows(P * 3), O=_rows(P * 4), g=P, s0=P, s1=P)
    a.update(kw)
    st = cf.lib().b2b_linear_attn_step(plan._h, a["batch"], a["Q"], a["K"], a["V"], a["O"], a["g"], a["s0"], a["s1"], None)
    assert st == status


def test_binding_checks_linear():
    plan = cf.LinearAttention("f16", 4, 2, 64)
    q, k, cu, g = _t(10, 4, 64), _t(10, 2, 64), _cu(0, 10), _t(4, dtype=torch.float32)
    s = _t(1, 4, 64, 64, dtype=torch.float32)
    for kw, match in [
        (dict(Q=q.float()), "Q: dtype"), (dict(K=k[:9]), "K: shape"), (dict(V=_t(10, 4, 64)), "V: shape"),
        (dict(log_decay=g[:3]), "log_decay"), (dict(log_decay=g.double()), "log_decay"), (dict(cu=cu.long()), "cu"),
        (dict(state=s.half()), "state"), (dict(state=_t(2, 4, 64, 64, dtype=torch.float32)), "state"),
        (dict(state_out=s.transpose(2, 3)), "state_out"), (dict(O=q[:3]), "O: shape"), (dict(), "device"),
    ]:
        a = dict(Q=q, K=k, V=k, log_decay=g, cu=cu)
        a.update(kw)
        with pytest.raises(ValueError, match=match):
            plan.run(**a)
    for kw, match in [(dict(state=None), "state"), (dict(state=s), "state"),
                      (dict(state=_t(10, 4, 64, 64, dtype=torch.float32)), "device")]:
        with pytest.raises(ValueError, match=match):
            plan.step(q, k, k, g, **kw)
    with pytest.raises(cf.B2BError, match="not supported"):
        cf.LinearAttention("f16", 4, 2, 96)


def test_usual_calls_leave_the_rest_to_python():
    """The compiled binding takes no call whose tensors are not on a device, and
    none of a plan that is closed; whatever it is given, it raises nothing."""
    from chip_fusion_amd import _attn
    plan, lin = cf.Attention("f16", 4, 2, 64), cf.LinearAttention("f16", 4, 2, 64)
    q, k, cu, g = _t(10, 4, 64), _t(10, 2, 64), _cu(0, 10), _t(4, dtype=torch.float32)
    u = plan._usual
    for args in [(q, k, k, cu, None, None, False), (q, k, k, cu, cu, q, True), (None,) * 7, (1, 2, 3, 4, 5, 6, 7), (q, k), (),
                 (q.numpy(), k, k, cu, None, None, False)]:
        assert u.attention(*args) is None and u.prefix(*args) is None and u.linear_step(*args) is None
        assert u.linear(*args) is None and u.linear(*args, None) is None
    assert lin._usual.linear(q, k, k, g, cu, None, None, None) is None
    plan.close()
    assert u.attention(q, k, k, cu, None, None, False) is None
    with pytest.raises(TypeError):
        _attn.Call(1, 2)
