"""The compiled calls of paged attention and rotations with stand-ins for tensors
and for the library's functions: which calls they take, what they launch, how
often, and what they leave to the checks in Python."""
import ctypes
import os
import subprocess
import sys

import pytest

import chip_fusion_amd as cf
from test_attention_calls_cpu import TORCH, Tensor

_attn = pytest.importorskip("chip_fusion_amd._attn")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(cf.__file__)))
H, KV, D, PAGE = 4, 2, 64, 16


class Strided(Tensor):
    """A stand-in with strides of its own."""

    def __init__(self, shape, dtype, stride):
        super().__init__(shape, dtype)
        self._stride = tuple(stride)

    def stride(self):
        return self._stride


class Plan:
    def __init__(self, status=0, refusal=0, axes=1, weights=1):
        self.runs = 0

        def run():
            self.runs += 1
            return status

        def workspace(plan, seqs, rows, width, out):
            out[0] = 64
            return refusal

        self.held = [ctypes.CFUNCTYPE(ctypes.c_int)(run),
                     ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                      ctypes.POINTER(ctypes.c_size_t))(workspace)]
        at, ws = (ctypes.cast(f, ctypes.c_void_p).value for f in self.held)
        self.call = _attn.Call(1, ws, at, at, H, KV, D, "f16", TORCH, cf._check, PAGE, axes, weights)


def _t(*shape, dtype="f16"):
    return Tensor(shape, dtype)


def _args(rows=5):
    q, k, v = _t(rows, H, D), _t(rows, KV, D), _t(rows, KV, D)
    kc, vc = _t(9, PAGE, KV, D), _t(9, PAGE, KV, D)
    return q, k, v, kc, vc, _t(rows, 3, dtype="i32"), _t(rows, dtype="i32"), _t(rows + 1, dtype="i32")


def _calls(p):
    q, k, v, kc, vc, table, lens, cu = _args()
    pos, w = _t(5, dtype="i32"), _t(D)
    return [("b2b_paged_attn_run", lambda: p.call.paged(q, kc, vc, table, lens, cu, None, True)),
            ("b2b_paged_attn_run", lambda: p.call.paged(q, kc, vc, table, lens, None, _t(5, H, D), False)),
            ("b2b_rotary_run", lambda: p.call.rotary(q, k, pos, w, None, None, None)),
            ("b2b_rotary_append", lambda: p.call.append(q, k, v, kc, vc, table, lens, cu, None, w, w, q))]


def test_a_run_is_made_once():
    p = Plan()
    for i, (name, call) in enumerate(_calls(p)):
        out = call()
        assert out is not None and p.runs == i + 1, name


@pytest.mark.parametrize("status", [1, 3])
def test_a_status_of_the_run_is_raised(status):
    p = Plan(status)
    for i, (name, call) in enumerate(_calls(p)):
        with pytest.raises(cf.B2BError, match=name) as e:
            call()
        assert e.value.status == status and p.runs == i + 1


def test_what_is_refused_before_the_run_is_left_to_python():
    p = Plan(0, 1)
    for name, call in _calls(p)[:2]:
        assert call() is None and p.runs == 0, name


def test_a_closed_call_makes_none():
    p = Plan()
    p.call.close()
    for name, call in _calls(p):
        assert call() is None and p.runs == 0, name


def test_what_is_not_usual_is_left_to_python():
    q, k, v, kc, vc, table, lens, cu = _args()
    pos, w, o = _t(5, dtype="i32"), _t(D), _t(5, H, D)
    odd = Strided((9, PAGE, KV, D), "f16", (PAGE * KV * D + 4, KV * D, D, 1))
    p = Plan()
    paged = [dict(q=_t(5, H, D, dtype="bf16")), dict(q=_t(4, H, D)), dict(kc=_t(9, 8, KV, D)), dict(vc=_t(8, PAGE, KV, D)),
             dict(kc=odd), dict(kc=_t(9, PAGE, KV + 1, D)), dict(table=_t(5, 3, dtype="i64")), dict(table=_t(4, 3, dtype="i32")),
             dict(table=Strided((5, 3), "i32", (1, 5))), dict(table=Strided((5, 3), "i32", (2, 1))), dict(lens=_t(4, dtype="i32")),
             dict(cu=_t(5, dtype="i32")), dict(o=_t(5, H, 32)), dict(lse=_t(5, H, dtype="f32")), dict(table=_t(5, 0, dtype="i32"))]
    for kw in paged:
        a = dict(q=q, kc=kc, vc=vc, table=table, lens=lens, cu=None, o=None, lse=False)
        a.update(kw)
        assert p.call.paged(*a.values()) is None, kw
    rotary = [dict(q=_t(4, H, D)), dict(k=_t(5, H, D)), dict(pos=None), dict(pos=_t(4, dtype="i32")), dict(pos=_t(5, dtype="i64")),
              dict(pos=_t(1, 5, dtype="i32")), dict(qw=_t(D, dtype="f32")), dict(kw=_t(D + 8)), dict(qo=_t(5, KV, D)),
              dict(ko=_t(5, H, D)), dict(q=Strided((5, H, D), "f16", (H * D + 8, D, 1)))]       # (its output is laid out in Python)
    for kw in rotary:
        a = dict(q=q, k=k, pos=pos, qw=w, kw=w, qo=None, ko=None)
        a.update(kw)
        assert p.call.rotary(*a.values()) is None, kw
    append = [dict(v=_t(5, H, D)), dict(vc=_t(9, 8, KV, D)), dict(kc=odd), dict(lens=_t(6, dtype="i32")), dict(pos=_t(4, dtype="i32"))]
    for kw in append:
        a = dict(q=q, k=k, v=v, kc=kc, vc=vc, table=table, lens=lens, cu=cu, pos=None, qw=None, kw=None, qo=o)
        a.update(kw)
        assert p.call.append(*a.values()) is None, kw
    assert p.runs == 0
    plain = Plan(weights=0)             # weights without a norm are refused in Python
    assert plain.call.rotary(q, k, pos, w, None, None, None) is None and plain.runs == 0
    assert plain.call.rotary(q, k, pos, None, None, None, None) is not None
    three = Plan(axes=3)
    assert three.call.rotary(q, k, pos, None, None, None, None) is None and three.runs == 0
    assert three.call.rotary(q, k, _t(2, 5, dtype="i32"), None, None, None, None) is None
    assert three.call.rotary(q, k, Strided((3, 5), "i32", (9, 1)), None, None, None, None) is not None


CALLS = """
import sys
sys.modules["chip_fusion_amd._attn"] = None          # as if the file were not there
import torch
import chip_fusion_amd as cf
t = lambda *shape: torch.zeros(shape, dtype=torch.float16)
i = lambda *shape: torch.zeros(shape, dtype=torch.int32)
q, k, c, rot = t(5, 4, 64), t(5, 2, 64), t(9, 16, 2, 64), cf.NormRotary("f16", 4, 2, 64)
for call in [lambda: cf.PagedAttention("f16", 4, 2, 64, 16).run(q, c, c, i(5, 3), i(5)), lambda: rot.run(q, k, i(5)),
             lambda: rot.append(q, k, k, c, c, i(5, 3), i(5))]:
    try:
        call()
    except ValueError as e:                          # all there is to say of them
        assert "a device (cuda) tensor is expected" in str(e), e
    else:
        raise AssertionError("host tensors accepted")
print("made in Python")
"""


def test_calls_without_the_compiled_binding():
    r = subprocess.run([sys.executable, "-c", CALLS], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "made in Python" in r.stdout, r.stderr[-2000:]


def test_the_binding_builds_without_torchs_headers(monkeypatch, tmp_path):
    """Then it looks at all tensors through their methods."""
    from chip_fusion_amd import build
    out = tmp_path / "_attn.so"
    monkeypatch.setattr(build, "PYATTN", str(out))
    monkeypatch.setattr(build, "_torch_flags", lambda: None)
    assert build.binding() == str(out) and out.exists()
    assert b"libtorch_python" not in out.read_bytes()
