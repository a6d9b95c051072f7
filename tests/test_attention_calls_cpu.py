"""The attention plans' compiled calls (pyattn.cpp) with stand-ins for tensors
and for the library's functions: what they launch, and how often."""
import ctypes
import types

import pytest

import chip_fusion_amd as cf

_attn = pytest.importorskip("chip_fusion_amd._attn")

H, KV, D = 4, 2, 64


class Tensor:
    def __init__(self, shape, dtype):
        self.shape, self.dtype = tuple(shape), dtype

    def stride(self):
        out, n = [], 1
        for m in reversed(self.shape):
            out.append(n)
            n *= m
        return tuple(reversed(out))

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x1000 + 16 * (id(self) & 0xFFFF)

    def new_empty(self, shape, dtype):
        return Tensor(shape if isinstance(shape, tuple) else (shape,), dtype)


TORCH = types.SimpleNamespace(
    Tensor=Tensor, float32="f32", int32="i32", uint8="u8", empty_like=lambda t: Tensor(t.shape, t.dtype),
    _C=types.SimpleNamespace(_cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda i: 0))


class Plan:
    """A compiled plan whose run and step return `status` and whose workspace
    call returns `refusal`; `runs` counts the former."""

    def __init__(self, status, refusal=0, three=False):
        self.runs = 0

        def run():
            self.runs += 1
            return status

        def workspace2(plan, seqs, rows, out):
            out[0] = 64
            return refusal

        def workspace3(plan, seqs, rows, keys, out):
            out[0] = 64
            return refusal

        size, i64 = ctypes.POINTER(ctypes.c_size_t), ctypes.c_int64
        # (a function that takes no arguments may be called with any)
        self.held = [ctypes.CFUNCTYPE(ctypes.c_int)(run),
                     ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_int32, i64, i64, size)(workspace3) if three
                     else ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_int32, i64, size)(workspace2)]
        at, ws = (ctypes.cast(f, ctypes.c_void_p).value for f in self.held)
        self.call = _attn.Call(1, ws, at, at, H, KV, D, "f16", TORCH, cf._check)


def _qkv(rows):
    return Tensor((rows, H, D), "f16"), Tensor((rows, KV, D), "f16"), Tensor((rows, KV, D), "f16")


def _calls(p3, p2):
    q, k, v = _qkv(5)
    own = Tensor((5, 9, KV, D), "f16")
    cu, lens, g = Tensor((2,), "i32"), Tensor((5,), "i32"), Tensor((H,), "f32")
    s1, s5 = Tensor((1, H, D, D), "f32"), Tensor((5, H, D, D), "f32")
    return [(p3, "b2b_attn_run", lambda: p3.call.attention(q, k, v, cu, None, None, True)),
            (p3, "b2b_prefix_attn_run", lambda: p3.call.prefix(q, k, v, own, own, lens, None)),
            (p2, "b2b_linear_attn_run", lambda: p2.call.linear(q, k, v, g, cu, s1, None, s1)),
            (p2, "b2b_linear_attn_step", lambda: p2.call.linear_step(q, k, v, g, s5, None, s5))]


def test_a_run_is_made_once():
    for plan, name, call in _calls(Plan(0, three=True), Plan(0)):
        before = plan.runs
        assert call() is not None and plan.runs == before + 1, name


@pytest.mark.parametrize("status", [1, 2, 5, 6])
def test_a_status_of_the_run_is_raised(status):
    """None would have the call made again, which takes a state in place twice
    if the first one was launched all the same."""
    for plan, name, call in _calls(Plan(status, three=True), Plan(status)):
        before = plan.runs
        with pytest.raises(cf.B2BError, match=name) as e:
            call()
        assert e.value.status == status and plan.runs == before + 1


def test_what_is_refused_before_the_run_is_left_to_python():
    """(A step asks for no workspace.)"""
    for plan, name, call in _calls(Plan(0, 1, three=True), Plan(0, 1))[:3]:
        assert call() is None and plan.runs == 0, name


@pytest.mark.parametrize("make,sizes", [
    (lambda: cf.Attention("f16", H, KV, D), (1, 4, 4096)), (lambda: cf.PrefixAttention("bf16", H, KV, D), (4, 100, 10)),
    (lambda: cf.LinearAttention("f16", H, KV, D), (1, 5000)),
])
@pytest.mark.parametrize("asked", [False, True])
def test_a_closed_plan_is_asked_for_nothing(make, sizes, asked):
    """Its memory is freed: sizes of a workspace, new ones and ones that it was
    asked for before, are an error."""
    plan = make()
    like = Tensor((1,), "f16")
    like.new_empty = lambda n, dtype: Tensor((n,), dtype)
    if asked:
        assert plan._workspaces.get(like, *sizes)[2] > 0
    plan.close()
    with pytest.raises(cf.B2BError):
        plan._workspaces.get(like, *sizes)
    plan.close()
