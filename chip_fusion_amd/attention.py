"""Attention plans (b2b_attn.h): argument checks and marshalling for the
library's attention kernels.

Tensors are taken as they lie: [rows, heads, dim] with any row and head
strides that are multiples of 8 elements, dim contiguous -- slices of a fused
projection, or [heads, rows, dim] storage seen transposed.  Everything runs
on the device that holds the tensors, on `stream` or on that device's current
stream (inputs made on another stream are the caller's to wait for and to
keep, as for torch's own operators); outputs and workspaces that a call
allocates come from torch's allocator on that stream, so overlapping calls
and captured graphs each have their own.  Forward only, as all of the
library: outputs carry no gradients.
"""
import ctypes

import torch

try:
    from . import _attn
except ImportError:         # a shortcut: every call is made in Python without it
    _attn = None
from . import ATTN_CAUSAL, DTYPES, Rows, TORCH_DTYPES, _check, lib

_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _heads3(t, name, dtype, rows, heads, dim):
    """As _rows for [rows, heads, dim] (rows None: any number): what nearly
    every call passes, in one look, the rest in _rows."""
    try:
        n, h, d = t.shape
        ld, hs, one = t.stride()
        p = t.data_ptr()
        if (t.dtype is dtype and p and n and h == heads and d == dim and (rows is None or n == rows)
                and one == 1 and ld >= dim and not (ld | hs | p >> 1) & 7):
            return Rows(p, ld, hs)
    except (AttributeError, TypeError, ValueError):
        pass
    return _rows(t, name, dtype, (rows, heads, dim))


def _rows(t, name, dtype, shape):
    """ValueError unless t is a tensor of that dtype and shape (None: any
    size) whose last three dimensions are rows of heads that the kernels can
    address; its b2b_rows_t."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a torch tensor is expected, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {dtype} expected, got {t.dtype}")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        want = ", ".join("any" if n is None else str(n) for n in shape)
        raise ValueError(f"{name}: shape [{want}] expected, got {list(t.shape)}")
    if t.numel() == 0:
        return Rows(None, 0, 0)
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    rows, heads, dim = t.shape[-3:]
    ld = t.stride(-3) if rows > 1 else dim      # a stride that is never stepped by
    hs = t.stride(-2) if heads > 1 else 0
    if ld % 8 or hs % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name}: rows and heads must start on 16-byte boundaries")
    if ld < dim:
        raise ValueError(f"{name}: rows overlap (row stride {ld}, {dim} columns)")
    return Rows(t.data_ptr(), ld, hs)


def _starts(cu, name, seqs=None):
    if not isinstance(cu, torch.Tensor) or cu.dtype is not torch.int32 or cu.dim() != 1 or not cu.is_contiguous():
        raise ValueError(f"{name}: a contiguous 1-D int32 tensor is expected")
    n = cu.numel() - 1
    if n < 0 or (seqs is not None and n != seqs):
        raise ValueError(f"{name}: {'at least one value' if seqs is None else f'{seqs + 1} values'} expected, "
                         f"got {n + 1}")
    return n


def _device_of(names, *tensors):
    """The CUDA device that holds all the tensors (None among them: not given)."""
    index = tensors[0].get_device()
    if index >= 0:
        for t in tensors:
            if t is not None and t.get_device() != index:
                break
        else:
            return index
    first = None
    for name, t in zip(names.split(), tensors):
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{name}: a device (cuda) tensor is expected, got one on {t.device}")
        if first is not None and t.device != first:
            raise ValueError(f"{name}: on {t.device}, the others on {first}")
        first = t.device


def _on(index, stream, call, *args):
    """call(handle, *args) with the tensors' device current and `stream` (or
    that device's current stream) the one that allocations belong to; handle:
    its hipStream_t."""
    if stream is None and _current_device() == index:
        return call(_raw_stream(index), *args)
    with torch.cuda.device(index):
        s = torch.cuda.current_stream() if stream is None else stream
        if s.device.index != index:
            raise ValueError(f"stream: on {s.device}, the tensors on cuda:{index}")
        with torch.cuda.stream(s):
            return call(s.cuda_stream, *args)


class _Workspaces:
    """Workspaces for one run each, from torch's allocator, which keeps one
    until the stream is past its run; the bytes that a call of some sizes needs
    are asked for once."""

    def __init__(self, call, handle):
        self._call, self._handle, self._bytes = call, handle, {}

    def close(self):
        """The plan is gone: asking is an error."""
        self._handle = None
        self._bytes.clear()

    def get(self, like, *sizes):
        """The workspace (a tensor, or None), its address and its bytes."""
        n = self._bytes.get(sizes)
        if n is None:
            out = ctypes.c_size_t()
            _check(self._call(self._handle, *sizes, ctypes.byref(out)), self._call.__name__)
            n = out.value
            if len(self._bytes) >= 4096:
                self._bytes.clear()
            self._bytes[sizes] = n
        if n == 0:
            return None, None, 0
        t = like.new_empty(n, dtype=torch.uint8)
        return t, t.data_ptr(), n


def _new(t):
    """An uninitialised dense tensor like t."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _ptr(t):
    return None if t is None else t.data_ptr()


class _NotCompiled:
    """Usual calls where there is no compiled binding: none."""

    def close(self):
        pass

    def attention(self, *args):
        return None

    prefix = linear = linear_step = attention


def _usual(handle, heads, kv_heads, dim, dtype, workspace, run, step=None):
    """The plan's usual calls (pyattn.cpp): on the current stream, tensors of the
    common layouts; they return None, with nothing launched, where the checks here
    are to be made."""
    if _attn is None:
        return _NotCompiled()
    at = lambda f: 0 if f is None else ctypes.cast(f, ctypes.c_void_p).value
    return _attn.Call(handle.value, at(workspace), at(run), at(step), heads, kv_heads, dim, dtype, torch, _check)


def _scale(scale):
    """A plan's scale in float32 (None: 0, the library's default)."""
    if scale is None:
        return 0.0
    value = ctypes.c_float(scale).value
    if not value > 0:
        raise ValueError("scale: a positive number (of float32) is expected")
    return value


class _Heads:
    """A plan of the attention of a model's heads (b2b_attn_create)."""

    def __init__(self, dtype, heads, kv_heads, head_dim, scale, flags):
        code = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
        scale = _scale(scale)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, head_dim
        h = ctypes.c_void_p()
        _check(lib().b2b_attn_create(ctypes.byref(h), code, heads, kv_heads, head_dim, scale, flags),
               "b2b_attn_create")
        self._h = h
        self.dtype = TORCH_DTYPES[code]
        self._call, workspace = getattr(lib(), self._run_call), getattr(lib(), self._workspace_call)
        self._workspaces = _Workspaces(workspace, h)
        self._usual = _usual(h, heads, kv_heads, head_dim, self.dtype, workspace, self._call)

    def close(self):
        if getattr(self, "_h", None):
            self._usual.close()
            self._workspaces.close()
            lib().b2b_attn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Attention(_Heads):
    """Attention over packed sequences (b2b_attn_run): softmax(scale Q.K^T).V
    for each sequence and head, causal (aligned to the last key) or full.

    scale: of the scores, dim ** -0.5 by default."""

    _run_call, _workspace_call = "b2b_attn_run", "b2b_attn_workspace"

    def __init__(self, dtype, heads, kv_heads, head_dim, causal=True, scale=None):
        super().__init__(dtype, heads, kv_heads, head_dim, scale, ATTN_CAUSAL if causal else 0)

    def run(self, Q, K, V, cu_q, cu_k=None, O=None, lse=False, stream=None):
        """Q [rows, heads, dim], K and V [keys, kv_heads, dim]; sequence s has
        rows cu_q[s] .. cu_q[s+1]-1 of Q and cu_k[s] .. cu_k[s+1]-1 of K and V
        (device int32; cu_k defaults to cu_q).  Returns O, or (O, LSE) with
        `lse` (True, or a float32 tensor [rows, heads] to write).  Rows that
        belong to no sequence are not written."""
        if stream is None:
            out = self._usual.attention(Q, K, V, cu_q, cu_k, O, lse)
            if out is not None:
                return out
        cu_k = cu_q if cu_k is None else cu_k
        seqs = _starts(cu_q, "cu_q")
        if cu_k is not cu_q:
            _starts(cu_k, "cu_k", seqs)
        dtype, heads, kv_heads, dim = self.dtype, self.heads, self.kv_heads, self.dim
        q = _heads3(Q, "Q", dtype, None, heads, dim)
        k = _heads3(K, "K", dtype, None, kv_heads, dim)
        rows, keys = Q.shape[0], K.shape[0]
        v = _heads3(V, "V", dtype, keys, kv_heads, dim)
        want = lse is not False and lse is not None
        LSE = lse if isinstance(lse, torch.Tensor) else None
        o = None if O is None else _heads3(O, "O", dtype, rows, heads, dim)
        if LSE is not None and (LSE.dtype != torch.float32 or LSE.shape != Q.shape[:2] or not LSE.is_contiguous()):
            raise ValueError("lse: a contiguous float32 tensor [rows, heads] is expected")
        index = _device_of("Q K V cu_q cu_k O lse", Q, K, V, cu_q, cu_k, O, LSE)
        return _on(index, stream, self._run, seqs, rows, keys, q, k, v, o, Q, O, cu_q, cu_k, want, LSE)

    def _run(self, stream, seqs, rows, keys, q, k, v, o, Q, O, cu_q, cu_k, want, LSE):
        if O is None:
            O = _new(Q)
            o = Rows(O.data_ptr(), self.heads * self.dim, self.dim)
        if want and LSE is None:
            LSE = Q.new_empty((rows, self.heads), dtype=torch.float32)
        keep, wp, n = self._workspaces.get(Q, seqs, rows, keys)
        st = self._call(self._h, seqs, rows, keys, q, k, v, o, cu_q.data_ptr(), cu_k.data_ptr(), _ptr(LSE), wp, n, stream)
        if st:
            _check(st, "b2b_attn_run")
        return (O, LSE) if want else O


class PrefixAttention(_Heads):
    """Attention of one new token a request, all requests behind one shared
    prefix (b2b_prefix_attn_run): the prefix is read once for the batch."""

    _run_call, _workspace_call = "b2b_prefix_attn_run", "b2b_prefix_attn_workspace"

    def __init__(self, dtype, heads, kv_heads, head_dim, scale=None):
        super().__init__(dtype, heads, kv_heads, head_dim, scale, 0)

    def run(self, Q, Kp, Vp, K, V, lens, O=None, stream=None):
        """Q [batch, heads, dim]; Kp, Vp [prefix, kv_heads, dim], the shared
        keys and values; K, V [batch, own, kv_heads, dim], of which request b
        has the first lens[b] (device int32).  Returns O [batch, heads, dim]."""
        if stream is None:
            out = self._usual.prefix(Q, Kp, Vp, K, V, lens, O)
            if out is not None:
                return out
        dtype, heads, kv_heads, dim = self.dtype, self.heads, self.kv_heads, self.dim
        q = _heads3(Q, "Q", dtype, None, heads, dim)
        batch = Q.shape[0]
        kp = _heads3(Kp, "Kp", dtype, None, kv_heads, dim)
        prefix = Kp.shape[0]
        vp = _heads3(Vp, "Vp", dtype, prefix, kv_heads, dim)
        k, ks = self._own(K, "K", batch, None)
        own = K.shape[1]
        v, vs = self._own(V, "V", batch, own)
        if not isinstance(lens, torch.Tensor) or lens.dtype is not torch.int32 or lens.shape != (batch,) \
                or not lens.is_contiguous():
            raise ValueError(f"lens: a contiguous int32 tensor [{batch}] is expected")
        o = None if O is None else _heads3(O, "O", dtype, batch, heads, dim)
        index = _device_of("Q Kp Vp K V lens O", Q, Kp, Vp, K, V, lens, O)
        return _on(index, stream, self._run, batch, prefix, own, q, kp, vp, k, ks, v, vs, o, Q, O, lens)

    def _own(self, t, name, batch, own):
        """Requests' own keys or values [batch, own, kv_heads, dim]: their
        b2b_rows_t and the stride from one request's to the next one's."""
        try:
            b, n, h, d = t.shape
            far, ld, hs, one = t.stride()
            p = t.data_ptr()
            if (t.dtype is self.dtype and p and n and b == batch and h == self.kv_heads and d == self.dim
                    and (own is None or n == own) and one == 1 and ld >= d and not (far | ld | hs | p >> 1) & 7):
                return Rows(p, ld, hs), far
        except (AttributeError, TypeError, ValueError):
            pass
        r = _rows(t, name, self.dtype, (batch, own, self.kv_heads, self.dim))
        far = t.stride(0) if batch > 1 and t.shape[1] else 0
        if far % 8:
            raise ValueError(f"{name}: requests must start on 16-byte boundaries")
        return r, far

    def _run(self, stream, batch, prefix, own, q, kp, vp, k, ks, v, vs, o, Q, O, lens):
        if O is None:
            O = _new(Q)
            o = Rows(O.data_ptr(), self.heads * self.dim, self.dim)
        keep, wp, n = self._workspaces.get(Q, batch, prefix, own)
        st = self._call(self._h, batch, prefix, own, q, kp, vp, k, ks, v, vs, lens.data_ptr(), o, wp, n, stream)
        if st:
            _check(st, "b2b_prefix_attn_run")
        return O


class LinearAttention:
    """Linear attention with a decay for each head (b2b_linear_attn_create):
    S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = scale q_t^T S_t, with
    float32 states [heads, dim, dim] (row: key element, column: value element).

    scale: dim ** -0.5 by default."""

    def __init__(self, dtype, heads, kv_heads, head_dim, scale=None):
        code = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
        scale = _scale(scale)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, head_dim
        h = ctypes.c_void_p()
        _check(lib().b2b_linear_attn_create(ctypes.byref(h), code, heads, kv_heads, head_dim, scale),
               "b2b_linear_attn_create")
        self._h = h
        self.dtype = TORCH_DTYPES[code]
        L = lib()
        self._workspaces = _Workspaces(L.b2b_linear_attn_workspace, h)
        self._usual = _usual(h, heads, kv_heads, head_dim, self.dtype, L.b2b_linear_attn_workspace, L.b2b_linear_attn_run,
                             L.b2b_linear_attn_step)

    def _operands(self, Q, K, V, log_decay, O):
        dtype, dim = self.dtype, self.dim
        q = _heads3(Q, "Q", dtype, None, self.heads, dim)
        rows = Q.shape[0]
        k = _heads3(K, "K", dtype, rows, self.kv_heads, dim)
        v = _heads3(V, "V", dtype, rows, self.kv_heads, dim)
        o = None if O is None else _heads3(O, "O", dtype, rows, self.heads, dim)
        if not isinstance(log_decay, torch.Tensor) or log_decay.dtype is not torch.float32 \
                or log_decay.shape != (self.heads,) or not log_decay.is_contiguous():
            raise ValueError(f"log_decay: a contiguous float32 tensor [{self.heads}] is expected")
        return rows, q, k, v, o

    def _state(self, t, name, n):
        if t is None:
            return
        want = (n, self.heads, self.dim, self.dim)
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.shape != want \
                or not t.is_contiguous() or t.data_ptr() % 16:
            raise ValueError(f"{name}: a contiguous, 16-byte aligned float32 tensor {list(want)} is expected")

    def run(self, Q, K, V, log_decay, cu, state=None, O=None, state_out=None, stream=None):
        """Prompts: Q [rows, heads, dim], K and V [rows, kv_heads, dim], rows
        cu[s] .. cu[s+1]-1 being sequence s (device int32); state: the states
        before them [seqs, heads, dim, dim] (zero by default).  Returns O and
        the states after them (state_out, which may be `state`)."""
        if stream is None:
            out = self._usual.linear(Q, K, V, log_decay, cu, state, O, state_out)
            if out is not None:
                return out
        rows, q, k, v, o = self._operands(Q, K, V, log_decay, O)
        seqs = _starts(cu, "cu")
        self._state(state, "state", seqs)
        self._state(state_out, "state_out", seqs)
        index = _device_of("Q K V log_decay cu state O state_out", Q, K, V, log_decay, cu, state, O, state_out)
        return _on(index, stream, self._run, seqs, rows, q, k, v, o, Q, O, log_decay, cu, state, state_out)

    def _run(self, stream, seqs, rows, q, k, v, o, Q, O, log_decay, cu, state, after):
        if O is None:
            O, o = self._new_out(Q)
        if after is None:
            after = Q.new_empty((seqs, self.heads, self.dim, self.dim), dtype=torch.float32)
        keep, wp, n = self._workspaces.get(Q, seqs, rows)
        st = lib().b2b_linear_attn_run(self._h, seqs, rows, q, k, v, o, log_decay.data_ptr(), cu.data_ptr(), _ptr(state),
                                       after.data_ptr(), wp, n, stream)
        if st:
            _check(st, "b2b_linear_attn_run")
        return O, after

    def step(self, Q, K, V, log_decay, state, O=None, state_out=None, stream=None):
        """One token of each request: row b of Q, K and V on state b
        [batch, heads, dim, dim].  Returns O and the states after it
        (state_out, which may be `state`)."""
        if stream is None:
            out = self._usual.linear_step(Q, K, V, log_decay, state, O, state_out)
            if out is not None:
                return out
        rows, q, k, v, o = self._operands(Q, K, V, log_decay, O)
        if state is None:
            raise ValueError("state: a tensor is expected")
        self._state(state, "state", rows)
        self._state(state_out, "state_out", rows)
        index = _device_of("Q K V log_decay state O state_out", Q, K, V, log_decay, state, O, state_out)
        return _on(index, stream, self._step, rows, q, k, v, o, Q, O, log_decay, state, state_out)

    def _step(self, stream, rows, q, k, v, o, Q, O, log_decay, state, after):
        if O is None:
            O, o = self._new_out(Q)
        if after is None:
            after = torch.empty_like(state)
        st = lib().b2b_linear_attn_step(self._h, rows, q, k, v, o, log_decay.data_ptr(), state.data_ptr(), after.data_ptr(),
                                        stream)
        if st:
            _check(st, "b2b_linear_attn_step")
        return O, after

    def _new_out(self, Q):
        O = _new(Q)
        return O, Rows(O.data_ptr(), self.heads * self.dim, self.dim)

    def close(self):
        if getattr(self, "_h", None):
            self._usual.close()
            self._workspaces.close()
            lib().b2b_linear_attn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
