"""Attention plans (b2b_attn.h): argument checks and marshalling for the
library's attention kernels: packed prompts (under a window or not), single
tokens behind a shared prefix, new tokens over a paged cache, linear attention,
and the norms and rotations of queries and keys before them.

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
from . import ATTN_CAUSAL, DTYPES, Pages, ROTARY_INTERLEAVED, ROTARY_NORM, Rows, TORCH_DTYPES, _check, lib

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

    prefix = linear = linear_step = paged = rotary = append = attention


def _usual(handle, heads, kv_heads, dim, dtype, workspace, run, step=None, page=0, axes=1, weights=False):
    """The plan's usual calls (pyattn.cpp): on the current stream, tensors of the
    common layouts; they return None, with nothing launched, where the checks here
    are to be made."""
    if _attn is None:
        return _NotCompiled()
    at = lambda f: 0 if f is None else ctypes.cast(f, ctypes.c_void_p).value
    return _attn.Call(handle.value, at(workspace), at(run), at(step), heads, kv_heads, dim, dtype, torch, _check, page,
                      axes, weights)


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

    _create_call = "b2b_attn_create"
    page_size = 0       # keys a page

    def __init__(self, dtype, heads, kv_heads, head_dim, *rest):
        """rest: what the create call takes after head_dim."""
        code = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, head_dim
        h = ctypes.c_void_p()
        _check(getattr(lib(), self._create_call)(ctypes.byref(h), code, heads, kv_heads, head_dim, *rest), self._create_call)
        self._h = h
        self.dtype = TORCH_DTYPES[code]
        self._call, workspace = getattr(lib(), self._run_call), getattr(lib(), self._workspace_call)
        self._workspaces = _Workspaces(workspace, h)
        self._usual = _usual(h, heads, kv_heads, head_dim, self.dtype, workspace, self._call, page=self.page_size)

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


def _window(window, sinks):
    """A window and its sinks as the library takes them (0: none)."""
    for name, n, least in (("window", 1 if window is None else window, 1), ("sinks", sinks, 0)):
        if isinstance(n, bool) or not isinstance(n, int) or not least <= n <= 1 << 30:
            raise ValueError(f"{name}: a whole number from {least} to 2^30 is expected, got {n!r}")
    if window is None and sinks:
        raise ValueError("sinks: without a window every earlier key is visible")
    return window or 0, sinks


class Attention(_Heads):
    """Attention over packed sequences (b2b_attn_run): softmax(scale Q.K^T).V
    for each sequence and head, causal (aligned to the last key) or full.

    scale: of the scores, dim ** -0.5 by default.
    window: causal rows see their last `window` keys only, and the sequence's
    first `sinks` (b2b_attn_create_window)."""

    _run_call, _workspace_call = "b2b_attn_run", "b2b_attn_workspace"

    def __init__(self, dtype, heads, kv_heads, head_dim, causal=True, scale=None, window=None, sinks=0):
        scale = _scale(scale)
        window, sinks = _window(window, sinks)
        if window:
            if not causal:
                raise ValueError("window: causal attention only")
            self._create_call = "b2b_attn_create_window"
            super().__init__(dtype, heads, kv_heads, head_dim, scale, window, sinks)
        else:
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
        super().__init__(dtype, heads, kv_heads, head_dim, _scale(scale), 0)

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


def _pages(t, name, dtype, pages, size, heads, dim):
    """ValueError unless t is a cache's pages [pages, size, heads, dim] that the
    kernels can address; its b2b_pages_t."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a torch tensor is expected, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {dtype} expected, got {t.dtype}")
    want = (pages, size, heads, dim)
    if t.dim() != 4 or any(n is not None and n != m for n, m in zip(want, t.shape)):
        raise ValueError(f"{name}: shape [{', '.join('any' if n is None else str(n) for n in want)}] expected, "
                         f"got {list(t.shape)}")
    if max(t.shape[:2]) >= 1 << 31:         # (the library's own checks see 32 bits)
        raise ValueError(f"{name}: fewer than 2^31 pages and keys a page are expected, got {list(t.shape)}")
    if t.numel() == 0:
        return Pages(None, 0, 0, 0)
    strides = [st if n > 1 else 0 for st, n in zip(t.stride(), t.shape)]      # 0: never stepped by
    if t.stride(3) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if any(st % 8 for st in strides[:3]) or t.data_ptr() % 16:
        raise ValueError(f"{name}: pages, rows and heads must start on 16-byte boundaries")
    return Pages(t.data_ptr(), *strides[:3])


def _ints(t, name, shape):
    """ValueError unless t is a contiguous int32 tensor of that shape."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 tensor {list(shape)} is expected")


def _table(table, lens, cu, rows):
    """The sequences, the table's width and its row stride."""
    if not isinstance(table, torch.Tensor) or table.dtype is not torch.int32 or table.dim() != 2 \
            or (table.shape[1] > 1 and table.stride(1) != 1) or (table.shape[0] > 1 and table.stride(0) < table.shape[1]):
        raise ValueError("table: an int32 tensor [seqs, width] with contiguous rows is expected")
    seqs, width = table.shape
    if max(seqs, width) >= 1 << 31:         # (the library's own checks see 32 bits)
        raise ValueError(f"table: fewer than 2^31 sequences and places are expected, got {list(table.shape)}")
    _ints(lens, "lens", (seqs,))
    if cu is not None:
        _starts(cu, "cu", seqs)
    elif rows != seqs:
        raise ValueError(f"cu: without it every sequence has one row, got {rows} rows and {seqs} sequences")
    return seqs, width, table.stride(0) if seqs > 1 else width


class PagedAttention(_Heads):
    """Causal attention of new tokens over a paged cache (b2b_paged_attn_run):
    one token of a sequence or a chunk of them, each sequence as it comes.

    page_size: keys a page, any number.
    window, sinks: as for Attention."""

    _create_call, _run_call, _workspace_call = "b2b_paged_attn_create", "b2b_paged_attn_run", "b2b_paged_attn_workspace"

    def __init__(self, dtype, heads, kv_heads, head_dim, page_size, scale=None, window=None, sinks=0):
        window, sinks = _window(window, sinks)
        self.page_size = page_size
        super().__init__(dtype, heads, kv_heads, head_dim, page_size, _scale(scale), window, sinks)

    def run(self, Q, K, V, table, lens, cu=None, O=None, lse=False, stream=None):
        """Q [rows, heads, dim]: rows cu[s] .. cu[s+1]-1 (device int32; None: row
        s) are the last tokens of sequence s, which has lens[s] keys with theirs.
        K, V [pages, page_size, kv_heads, dim], any strides that are multiples of
        8; key j of sequence s is in page table[s, j // page_size] (device int32
        [seqs, width]).  Returns O, or (O, LSE) with `lse` (True, or a float32
        tensor [rows, heads] to write).  Rows that belong to no sequence are
        not written."""
        if stream is None:
            out = self._usual.paged(Q, K, V, table, lens, cu, O, lse)
            if out is not None:
                return out
        dtype, heads, kv_heads, dim = self.dtype, self.heads, self.kv_heads, self.dim
        q = _heads3(Q, "Q", dtype, None, heads, dim)
        rows = Q.shape[0]
        k = _pages(K, "K", dtype, None, self.page_size, kv_heads, dim)
        v = _pages(V, "V", dtype, K.shape[0], self.page_size, kv_heads, dim)
        seqs, width, table_ld = _table(table, lens, cu, rows)
        want = lse is not False and lse is not None
        LSE = lse if isinstance(lse, torch.Tensor) else None
        o = None if O is None else _heads3(O, "O", dtype, rows, heads, dim)
        if LSE is not None and (LSE.dtype != torch.float32 or LSE.shape != Q.shape[:2] or not LSE.is_contiguous()):
            raise ValueError("lse: a contiguous float32 tensor [rows, heads] is expected")
        index = _device_of("Q K V table lens cu O lse", Q, K, V, table, lens, cu, O, LSE)
        return _on(index, stream, self._run, seqs, rows, q, k, v, K.shape[0], table, width, table_ld, lens, cu, o, Q, O, want,
                   LSE)

    def _run(self, stream, seqs, rows, q, k, v, pages, table, width, table_ld, lens, cu, o, Q, O, want, LSE):
        if O is None:
            O = _new(Q)
            o = Rows(O.data_ptr(), self.heads * self.dim, self.dim)
        if want and LSE is None:
            LSE = Q.new_empty((rows, self.heads), dtype=torch.float32)
        keep, wp, n = self._workspaces.get(Q, seqs, rows, width)
        st = self._call(self._h, seqs, rows, q, k, v, pages, table.data_ptr(), width, table_ld, lens.data_ptr(), _ptr(cu), o,
                        _ptr(LSE), wp, n, stream)
        if st:
            _check(st, "b2b_paged_attn_run")
        return (O, LSE) if want else O


class NormRotary:
    """Norms of queries and keys for each head and their rotation by the
    position, in one pass (b2b_rotary_create), and the same for new tokens
    whose keys and values go into the pages of a cache.

    rotary_dim: how many of a head's first elements turn (all by default; 0: none).
    base, freqs: pair i turns by freqs[i] radians a position, base ** (-2 i /
    rotary_dim) by default.
    sections: how many of the pairs, in order, follow each axis of the positions
    (time, height, width ...); or axes_of: every pair's axis.
    interleaved: pair i is elements 2i and 2i + 1 (else i and i + rotary_dim / 2).
    eps: of the norm; None: no norm."""

    def __init__(self, dtype, heads, kv_heads, head_dim, rotary_dim=None, base=10000.0, freqs=None, sections=None, axes_of=None,
                 interleaved=False, eps=1e-6):
        code = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if not isinstance(rotary_dim, int) or rotary_dim < 0:
            raise ValueError(f"rotary_dim: a whole number from 0 is expected, got {rotary_dim!r}")
        pairs = rotary_dim // 2
        if freqs is None:
            if not base > 0:
                raise ValueError("base: a positive number is expected")
            freqs = [base ** (-2.0 * i / rotary_dim) for i in range(pairs)]
        freqs = [float(f) for f in freqs]
        if len(freqs) != pairs:
            raise ValueError(f"freqs: {pairs} values expected, got {len(freqs)}")
        if sections is not None:
            if axes_of is not None:
                raise ValueError("axes_of: either it or sections")
            if any(n < 0 for n in sections) or sum(sections) != pairs:
                raise ValueError(f"sections: {pairs} pairs in all expected, got {list(sections)}")
            axes_of = [axis for axis, n in enumerate(sections) for _ in range(n)]
        elif axes_of is None:
            axes_of = [0] * pairs
        axes_of = [int(x) for x in axes_of]
        if len(axes_of) != pairs:
            raise ValueError(f"axes_of: {pairs} values expected, got {len(axes_of)}")
        axes = len(sections) if sections else max(axes_of, default=0) + 1
        flags = (0 if eps is None else ROTARY_NORM) | (ROTARY_INTERLEAVED if interleaved else 0)
        h = ctypes.c_void_p()
        _check(lib().b2b_rotary_create(ctypes.byref(h), code, heads, kv_heads, head_dim, rotary_dim,
                                       (ctypes.c_double * pairs)(*freqs), (ctypes.c_int * pairs)(*axes_of), axes,
                                       0.0 if eps is None else eps, flags), "b2b_rotary_create")
        self._h = h
        self.dtype = TORCH_DTYPES[code]
        self.heads, self.kv_heads, self.dim, self.rotary_dim, self.axes, self.norm = \
            heads, kv_heads, head_dim, rotary_dim, axes, eps is not None
        self._usual = _usual(h, heads, kv_heads, head_dim, self.dtype, None, lib().b2b_rotary_run, lib().b2b_rotary_append,
                             axes=axes, weights=self.norm)

    def _common(self, Q, K, positions, q_weight, k_weight, Q_out):
        dtype, dim = self.dtype, self.dim
        q = _heads3(Q, "Q", dtype, None, self.heads, dim)
        rows = Q.shape[0]
        k = _heads3(K, "K", dtype, rows, self.kv_heads, dim)
        qo = None if Q_out is None else _heads3(Q_out, "Q_out", dtype, rows, self.heads, dim)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is None:
                continue
            if not self.norm:
                raise ValueError(f"{name}: the plan has no norm")
            if not isinstance(w, torch.Tensor) or w.dtype is not dtype or w.shape != (dim,) or not w.is_contiguous() \
                    or w.data_ptr() % 16:
                raise ValueError(f"{name}: a contiguous, 16-byte aligned {dtype} tensor [{dim}] is expected")
        far = 0
        if positions is not None:
            if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int32 \
                    or positions.shape != ((rows,) if self.axes == 1 and positions.dim() == 1 else (self.axes, rows)) \
                    or (rows > 1 and positions.stride(-1) != 1):
                want = f"[{rows}] or [1, {rows}]" if self.axes == 1 else f"[{self.axes}, {rows}]"
                raise ValueError(f"positions: an int32 tensor {want} with contiguous rows is expected")
            far = positions.stride(0) if self.axes > 1 else rows
        return rows, q, k, qo, far

    def run(self, Q, K, positions=None, q_weight=None, k_weight=None, Q_out=None, K_out=None, stream=None):
        """Q [rows, heads, dim], K [rows, kv_heads, dim]; positions: device int32
        [rows], or [axes, rows] with several axes (None only where rotary_dim is
        0); weights: [dim], 1 by default.  Returns Q_out and K_out, which may be
        Q and K."""
        if stream is None:
            out = self._usual.rotary(Q, K, positions, q_weight, k_weight, Q_out, K_out)
            if out is not None:
                return out
        rows, q, k, qo, far = self._common(Q, K, positions, q_weight, k_weight, Q_out)
        if positions is None and self.rotary_dim:
            raise ValueError("positions: a tensor is expected")
        ko = None if K_out is None else _heads3(K_out, "K_out", self.dtype, rows, self.kv_heads, self.dim)
        index = _device_of("Q K positions q_weight k_weight Q_out K_out", Q, K, positions, q_weight, k_weight, Q_out, K_out)
        return _on(index, stream, self._run, rows, q, k, qo, ko, positions, far, q_weight, k_weight, Q, K, Q_out, K_out)

    def _run(self, stream, rows, q, k, qo, ko, positions, far, q_weight, k_weight, Q, K, Q_out, K_out):
        if Q_out is None:
            Q_out = _new(Q)
            qo = Rows(Q_out.data_ptr(), self.heads * self.dim, self.dim)
        if K_out is None:
            K_out = _new(K)
            ko = Rows(K_out.data_ptr(), self.kv_heads * self.dim, self.dim)
        st = lib().b2b_rotary_run(self._h, rows, q, k, qo, ko, _ptr(positions), far, _ptr(q_weight), _ptr(k_weight), stream)
        if st:
            _check(st, "b2b_rotary_run")
        return Q_out, K_out

    def append(self, Q, K, V, k_cache, v_cache, table, lens, cu=None, positions=None, q_weight=None, k_weight=None,
               Q_out=None, stream=None):
        """New tokens: rows cu[s] .. cu[s+1]-1 (None: row s) of Q, K and V are the
        last ones of sequence s, which has lens[s] keys with theirs.  Their keys,
        normed and turned, and their values are written into the pages k_cache
        and v_cache [pages, page_size, kv_heads, dim] at the rows' places, where
        PagedAttention.run finds them with the same table, lens and cu.
        positions: the rows' places in their sequences by default.  Returns Q_out,
        which may be Q."""
        if stream is None:
            out = self._usual.append(Q, K, V, k_cache, v_cache, table, lens, cu, positions, q_weight, k_weight, Q_out)
            if out is not None:
                return out
        rows, q, k, qo, far = self._common(Q, K, positions, q_weight, k_weight, Q_out)
        v = _heads3(V, "V", self.dtype, rows, self.kv_heads, self.dim)
        kc = _pages(k_cache, "k_cache", self.dtype, None, None, self.kv_heads, self.dim)
        pages, size = k_cache.shape[:2]
        vc = _pages(v_cache, "v_cache", self.dtype, pages, size, self.kv_heads, self.dim)
        if size < 1:
            raise ValueError("k_cache: a page holds at least one key")
        seqs, width, table_ld = _table(table, lens, cu, rows)
        index = _device_of("Q K V k_cache v_cache table lens cu positions q_weight k_weight Q_out", Q, K, V, k_cache, v_cache,
                           table, lens, cu, positions, q_weight, k_weight, Q_out)
        return _on(index, stream, self._append, seqs, rows, q, k, v, qo, kc, vc, pages, size, table, width, table_ld, lens, cu,
                   positions, far, q_weight, k_weight, Q, Q_out)

    def _append(self, stream, seqs, rows, q, k, v, qo, kc, vc, pages, size, table, width, table_ld, lens, cu, positions, far,
                q_weight, k_weight, Q, Q_out):
        if Q_out is None:
            Q_out = _new(Q)
            qo = Rows(Q_out.data_ptr(), self.heads * self.dim, self.dim)
        st = lib().b2b_rotary_append(self._h, seqs, rows, q, k, v, qo, kc, vc, pages, size, table.data_ptr(), width, table_ld,
                                     lens.data_ptr(), _ptr(cu), _ptr(positions), far, _ptr(q_weight), _ptr(k_weight), stream)
        if st:
            _check(st, "b2b_rotary_append")
        return Q_out

    def close(self):
        if getattr(self, "_h", None):
            self._usual.close()
            lib().b2b_rotary_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


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
