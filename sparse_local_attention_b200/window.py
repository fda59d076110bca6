"""Causal sliding-window attention with sinks over token sequences.

The one-dimensional counterpart of sliding tile attention, for models that
produce their tokens in order: a query sees the last ``window`` tokens up to
its own and the first ``sinks`` tokens of its sequence.  Argument marshalling
for sta_window_forward / sta_window_backward of include/sta.h, which state the
semantics; the work runs in the CUDA kernels of libsta.so.
"""
from __future__ import annotations

import contextlib
import copy
import ctypes
import functools
import threading
import weakref
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from .sta import STA_CALL_CHECK, _check, _Rows, lib, refuse_tangents

STA_PACKED_ZERO = 0x4
STA_TYPE_BF16, STA_TYPE_FP16, STA_TYPE_E4M3, STA_TYPE_INT8 = 0, 1, 2, 3
IO_TYPES = {torch.bfloat16: STA_TYPE_BF16, torch.float16: STA_TYPE_FP16}


class _WindowProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "heads", "kv_heads", "head_dim", "q_len", "kv_len", "q_rows",
                                              "kv_rows", "window", "sinks", "type")] + [("scale", ctypes.c_float)]


def _rows(t: torch.Tensor) -> _Rows:
    b, h, r, _ = t.stride()
    return _Rows(t.data_ptr(), b, h, r)


def _in_place(t: torch.Tensor) -> bool:
    """Whether the kernels can address the tensor's rows where they are:
    contiguous rows, 16-byte aligned, at positive strides that are multiples
    of 8 elements (a stride of an extent of one is not used)."""
    b, h, r, e = t.stride()
    if e != 1 or t.data_ptr() & 15:
        return False
    if b > 0 and h > 0 and r > 0 and not (b | h | r) & 7:
        return True
    return all(n <= 1 or (s > 0 and s % 8 == 0) for n, s in zip(t.shape, (b, h, r)))


def _input(t: torch.Tensor, name: str, shape, dtype, device) -> torch.Tensor:
    """An input of [batch, heads, rows, d]: read in place if its strides allow it, else copied."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_cuda:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {device}, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")
    return t if _in_place(t) else t.clone(memory_format=torch.contiguous_format)


def _output(t: torch.Tensor, name: str, shape, dtype, device) -> torch.Tensor:
    if _input(t, name, shape, dtype, device) is not t:
        raise ValueError(f"{name}: expected 16-byte aligned rows at strides of multiples of 8, got strides {t.stride()}")
    return t


def _flat(t: Optional[torch.Tensor], name: str, shape, dtype, device) -> Optional[torch.Tensor]:
    """A contiguous device tensor of exactly this shape (int32 tables, fp32 statistics), or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        if stream.device != device:
            raise ValueError(f"stream of {stream.device} for tensors on {device}")
        with torch.cuda.stream(stream):
            yield


def _on(device, stream):
    """Context of a call: the tensors' device is current, and so is `stream` if
    one is given, so that what the call allocates belongs to it."""
    if stream is None and torch._C._cuda_getDevice() == device.index:
        return _HERE
    return _switched(device, stream)


_HERE = contextlib.nullcontext()


def _current_stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _int32(n, name: str) -> int:
    """n as the C call takes it: an int32 argument would lose the bits above."""
    n = int(n)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name}: expected a 32-bit integer, got {n}")
    return n


def _at(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _scratch(workspace: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {device}")
    return workspace


def _new(like: torch.Tensor) -> torch.Tensor:
    """An output laid out as `like`."""
    t = torch.empty_like(like)
    return t if _in_place(t) else torch.empty_like(like, memory_format=torch.contiguous_format)


def _statistics(shape, device) -> torch.Tensor:
    """An fp32 tensor of [batch, heads, rows]."""
    _, h, n = shape
    return torch.empty_strided(shape, (h * n, n, 1), dtype=torch.float32, device=device)


@functools.lru_cache(maxsize=64)
def _status(device) -> torch.Tensor:
    """The workspace of forward calls whose status nobody reads: its only word is
    written where a wait of the kernels runs out, which `check` reports."""
    return torch.empty(256, dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=256)
def _sized(batch, heads, kv_heads, head_dim, q_len, kv_len, q_rows, kv_rows, window, sinks, dtype, scale):
    """(problem, forward bytes, backward bytes) of one problem."""
    p = _WindowProblem(batch, heads, kv_heads, head_dim, q_len, kv_len, q_rows, kv_rows, window, sinks, dtype, scale)
    fwd, bwd = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().sta_window_workspace_size(ctypes.byref(p), ctypes.byref(fwd), ctypes.byref(bwd)),
           "sta_window_workspace_size")
    return p, fwd.value, bwd.value


class _Call:
    """The checked arguments that the forward and backward of one problem share."""

    def __init__(self, q, k, v, window, sinks, scale, cu_q, cu_kv, max_q, max_kv):
        for t, name in ((q, "q"), (k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
            if t.dim() != 4:
                raise ValueError(f"{name}: expected [batch, heads, rows, head_dim], got {tuple(t.shape)}")
        if q.dtype not in IO_TYPES:
            raise ValueError(f"q: expected bfloat16 or float16, got {q.dtype}")
        if (cu_q is None) != (cu_kv is None):
            raise ValueError("cu_q and cu_kv go together")
        self.dtype, self.device = dtype, device = q.dtype, q.device
        self.q_shape = batch, heads, nq, d = tuple(q.shape)
        _, kv_heads, nk, _ = k.shape
        self.kv_shape = batch, kv_heads, nk, d
        self.q = _input(q, "q", self.q_shape, dtype, device)
        self.k = _input(k, "k", self.kv_shape, dtype, device)
        self.v = _input(v, "v", self.kv_shape, dtype, device)
        self.packed = cu_q is not None
        self.cu_q, self.cu_kv = cu_q, cu_kv
        window, sinks = _int32(window, "window"), _int32(sinks, "sinks")
        if self.packed:
            if batch != 1:
                raise ValueError("packed sequences: expected a batch of 1")
            if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or not cu_q.numel():
                raise ValueError("cu_q: expected int32 [sequences + 1]")
            batch = cu_q.numel() - 1
            _flat(cu_q, "cu_q", (batch + 1,), torch.int32, q.device)
            _flat(cu_kv, "cu_kv", (batch + 1,), torch.int32, q.device)
            rows = (nq, nk)
            nq, nk = min(int(max_q) or nq, nq), min(int(max_kv) or nk, nk)
        else:
            rows = (0, 0)
        self.empty = 0 in self.q_shape or (self.packed and batch == 0)
        if self.empty and d not in (64, 128):  # other calls learn it from the library
            raise ValueError(f"q: expected a head_dim of 64 or 128, got {d}")
        # no key rows: queries see nothing.  The packed form still has to tell
        # the rows of its sequences from the rest, over a key row that none owns.
        self.no_keys = 0 in self.kv_shape
        if self.packed and self.no_keys and kv_heads and not self.empty:
            self.k = self.v = q.new_zeros((1, kv_heads, 1, d))
            self.no_keys = False
        if not self.empty:
            self.problem, self.fwd_bytes, self.bwd_bytes = _sized(
                batch, heads, kv_heads, d, nq, nk, *rows, window, sinks, IO_TYPES[dtype], float(scale))


def _forward(c: _Call, o=None, lse=None, workspace=None, check=False, want_lse=True):
    new = []
    if o is None:
        o = _new(c.q)
        new.append((o, 0.0))
    else:
        _output(o, "o", c.q_shape, c.dtype, c.device)
    if lse is None and want_lse:
        lse = _statistics(c.q_shape[:3], c.device)
        new.append((lse, float("-inf")))
    else:
        _flat(lse, "lse", c.q_shape[:3], torch.float32, c.device)
    flags = STA_CALL_CHECK if check else 0
    if c.packed:  # rows outside every sequence are not written
        if len(new) == 1 + (lse is not None) and not c.empty:
            flags |= STA_PACKED_ZERO
        else:
            for t, value in new:
                t.fill_(value)
    if not c.empty:
        if c.no_keys:
            o.zero_()
            if lse is not None:
                lse.fill_(float("-inf"))
            return o, lse
        ws = (_status(c.device) if workspace is None and not check and c.fwd_bytes <= 256 else
              _scratch(workspace, c.fwd_bytes, c.device))
        st = lib().sta_window_forward(ctypes.byref(c.problem), _rows(c.q), _rows(c.k), _rows(c.v), _rows(o), _at(lse),
                                      _at(c.cu_q), _at(c.cu_kv), ws.data_ptr(), ws.nbytes,
                                      _current_stream(c.device), flags)
        _check(st, "sta_window_forward")
    return o, lse


def _backward(c: _Call, o, lse, dout, dq=None, dk=None, dv=None, workspace=None, check=False):
    o = _input(o, "o", c.q_shape, c.dtype, c.device)
    dout = _input(dout, "dout", c.q_shape, c.dtype, c.device)
    _flat(lse, "lse", c.q_shape[:3], torch.float32, c.device)
    outs, new = [], []
    for t, like, shape, name in ((dq, c.q, c.q_shape, "dq"), (dk, c.k, c.kv_shape, "dk"), (dv, c.v, c.kv_shape, "dv")):
        outs.append(_output(t, name, shape, c.dtype, c.device) if t is not None else
                    _new(like) if like.shape == shape else like.new_empty(shape))
        if t is None:
            new.append(outs[-1])
    dq, dk, dv = outs
    flags = STA_CALL_CHECK if check else 0
    if c.packed and new:  # rows outside every sequence are not written
        if len(new) == 3 and not c.empty:
            flags |= STA_PACKED_ZERO
        else:
            torch._foreach_zero_(new)
    if c.empty or c.no_keys:
        if not c.packed:
            torch._foreach_zero_(outs)
        return dq, dk, dv
    dk_rows, dv_rows = (_rows(t if 0 not in c.kv_shape else torch.empty_like(c.k)) for t in (dk, dv))
    ws = _scratch(workspace, c.bwd_bytes, c.device)
    st = lib().sta_window_backward(ctypes.byref(c.problem), _rows(c.q), _rows(c.k), _rows(c.v), _rows(o), _at(lse),
                                   _rows(dout), _rows(dq), dk_rows, dv_rows, _at(c.cu_q), _at(c.cu_kv),
                                   ws.data_ptr(), ws.nbytes, _current_stream(c.device), flags)
    _check(st, "sta_window_backward")
    return dq, dk, dv


def _device_of(q) -> torch.device:
    if not isinstance(q, torch.Tensor):
        raise TypeError(f"q: expected a torch.Tensor, got {type(q).__name__}")
    if not q.is_cuda:
        raise ValueError(f"q: expected a CUDA tensor, got one on {q.device}")
    return q.device


def window_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int = 0, sinks: int = 0,
                   scale: float = 0.0, cu_q: Optional[torch.Tensor] = None, cu_kv: Optional[torch.Tensor] = None,
                   max_q: int = 0, max_kv: int = 0, o: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None,
                   check: bool = False, want_lse: bool = True):
    """(o, lse) of sliding-window attention with sinks.

    q [batch, heads, Nq, d], k and v [batch, kv_heads, Nk, d], bf16 or fp16, d
    64 or 128, kv_heads a divisor of heads; query row i sits at position
    i + Nk - Nq.  window 0: no limit.  Any strides with contiguous, 16-byte
    aligned rows are read in place; other inputs are copied first.  Not
    differentiable by itself: sliding_window_attention is.

    Packed sequences: a batch of 1 whose rows [cu[b], cu[b + 1]) hold sequence
    b (cu_q, cu_kv: int32 device tensors); max_q and max_kv are bounds on the
    sequences' lengths (default: the rows there are; longer sequences are cut).
    Work is laid out for every sequence up to the bounds, so pass them where there
    are many (64 documents of 512 tokens: forward and backward 0.9 ms with bounds
    and 6.4 without; 256: 3.4 and 93).
    Rows outside every sequence are left as they were in an `o` or `lse` that
    is passed in, and 0 (-inf) in a new one."""
    with _on(_device_of(q), stream):
        return _forward(_Call(q, k, v, window, sinks, scale, cu_q, cu_kv, max_q, max_kv), o, lse, workspace, check,
                        want_lse)


def window_backward(q, k, v, o, lse, dout, window: int = 0, sinks: int = 0, scale: float = 0.0, cu_q=None, cu_kv=None,
                    max_q: int = 0, max_kv: int = 0, dq=None, dk=None, dv=None, workspace=None, stream=None,
                    check: bool = False):
    """(dq, dk, dv) of window_forward from its inputs, its o and lse, and the
    gradient of o.  dk and dv sum over the query heads that share a key head."""
    with _on(_device_of(q), stream):
        return _backward(_Call(q, k, v, window, sinks, scale, cu_q, cu_kv, max_q, max_kv), o, lse, dout, dq, dk, dv,
                         workspace, check)


# The live graphs, each of which notes its stream and its leaves (by identity: it
# keeps them alive).  Nothing is kept on the leaves, which are saved and copied.
_graphs = weakref.WeakSet()
_graphs_lock = threading.Lock()


def _note_uses(ctx, tensors, stream: int):
    """Remember that the graph of `ctx` was built on `stream` over these leaves,
    or views of leaves.

    A gradient that is accumulated into a leaf runs on the stream on which the
    leaf was first used for as long as a graph of that use lives.  A backward
    pass captured on another stream would have to join that stream, which ends
    the capture and the process, so such a capture is refused."""
    used = [t if t.is_leaf else t._base for t, needed in zip(tensors, ctx.needs_input_grad) if needed]
    leaves = {id(t) for t in used if t is not None and t.is_leaf and t.requires_grad}
    if not leaves:
        return
    ctx.stream, ctx.leaves = stream, leaves
    with _graphs_lock:
        if torch.cuda.is_current_stream_capturing() and any(g.stream != stream and g.leaves & leaves for g in _graphs):
            raise RuntimeError("sliding_window_attention: an eager graph of the same leaf tensors is still alive; "
                               "release it (and its outputs) before capturing, or capture on detached leaves")
        _graphs.add(ctx)


class _SlidingWindowAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, args):
        with _on(q.device, None):
            _note_uses(ctx, (q, k, v), _current_stream(q.device))
            c = _Call(q, k, v, *args)
            o, lse = _forward(c)
        # autograd's to keep, to let go after the backward, and to refuse where
        # they have been written to in between
        ctx.save_for_backward(c.q, c.k, c.v, o, lse, c.cu_q, c.cu_kv)
        c.q = c.k = c.v = c.cu_q = c.cu_kv = None
        ctx.call = c
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        c = copy.copy(ctx.call)
        c.q, c.k, c.v, o, lse, c.cu_q, c.cu_kv = ctx.saved_tensors
        with _on(o.device, None):
            dq, dk, dv = _backward(c, o, lse, dout)
        return dq, dk, dv, None


def sliding_window_attention(q, k, v, window: int = 0, sinks: int = 0, scale: float = 0.0, cu_q=None, cu_kv=None,
                             max_q: int = 0, max_kv: int = 0) -> torch.Tensor:
    """window_forward's o, differentiable: when q, k or v requires a gradient
    the backward is one sta_window_backward call.  Shared key heads and
    broadcast inputs get the sum of their gradients."""
    refuse_tangents("sliding_window_attention", q, k, v)
    args = (window, sinks, scale, cu_q, cu_kv, max_q, max_kv)
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (q, k, v)):
        device = _device_of(q)
        with _on(device, None):
            return _SlidingWindowAttention.apply(q, k, v, args)
    return window_forward(q, k, v, *args, want_lse=False)[0]
