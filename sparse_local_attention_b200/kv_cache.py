"""A paged key/value cache in 8 bits: written, read back and attended to.

Argument marshalling for sta_cache_write / sta_cache_read /
sta_cache_attention of include/sta.h, which state the semantics.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .sta import STA_CALL_CHECK, _check, lib
from .window import (IO_TYPES, STA_TYPE_E4M3, STA_TYPE_INT8, _at, _current_stream, _flat, _input, _int32, _new, _on,
                     _output, _rows, _statistics)

STA_READ_ZERO = 0x2
CACHE_TYPES = {torch.float8_e4m3fn: STA_TYPE_E4M3, torch.int8: STA_TYPE_INT8}
BLOCKS, HEAD_DIMS = (16, 32, 64, 128), (64, 128)


def _check_sizes(pages: int, kv_heads: int, page_size: int, head_dim: int, block: int):
    """The sizes that the calls take."""
    if head_dim not in HEAD_DIMS:
        raise ValueError(f"head_dim: expected 64 or 128, got {head_dim}")
    if block not in BLOCKS:
        raise ValueError(f"block: expected 16, 32, 64 or 128 tokens per scale, got {block}")
    if page_size < 1 or page_size % block:
        raise ValueError(f"block {block} does not divide page_size {page_size}")
    if pages < 1 or not 1 <= kv_heads <= 65535 or pages * page_size >= 2 ** 31:
        raise ValueError(f"expected pages and kv_heads (up to 65535) above 0 and pages * page_size below 2^31, got {pages} "
                         f"pages of {page_size} tokens and {kv_heads} heads")


class _Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("pages", "kv_heads", "page_size", "block", "head_dim", "type")] + [
        (n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]


class KVCache:
    """`pages` pages of `page_size` tokens: codes k, v [pages, kv_heads,
    page_size, head_dim] (float8_e4m3fn or int8) and fp32 scales k_scale,
    v_scale [pages, kv_heads, page_size / block], one for every `block` tokens
    of a page and head.  A code c stands for c times its scale.

    Sequences own pages through a page table (int32 [batch, table_pages], the
    page of each page_size tokens; entries outside [0, pages) are absent pages),
    which the caller keeps, as well as the number of tokens of each sequence.
    head_dim: 64 or 128; block: 16, 32, 64 or 128, a divisor of page_size.
    One call may not write a page for two sequences, nor twice for one."""

    def __init__(self, pages: int, kv_heads: int, page_size: int, head_dim: int, block: int = 64,
                 dtype: torch.dtype = torch.float8_e4m3fn, device="cuda"):
        if dtype not in CACHE_TYPES:
            raise ValueError(f"dtype: expected float8_e4m3fn or int8, got {dtype}")
        _check_sizes(pages, kv_heads, page_size, head_dim, block)
        codes, scales = (pages, kv_heads, page_size, head_dim), (pages, kv_heads, page_size // block)
        zeros = [torch.zeros(codes, dtype=torch.uint8, device=device).view(dtype) for _ in range(2)]
        self._take(*zeros, *(torch.zeros(scales, dtype=torch.float32, device=device) for _ in range(2)))

    @classmethod
    def from_tensors(cls, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor) -> "KVCache":
        """A cache over existing codes and scales (not copied)."""
        self = cls.__new__(cls)
        self._take(k, v, k_scale, v_scale)
        return self

    def _take(self, k, v, k_scale, v_scale):
        for t, name in ((k, "k"), (v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if k.dim() != 4 or k_scale.dim() != 3 or k.dtype not in CACHE_TYPES or not k.is_cuda:
            raise ValueError(f"k: expected float8_e4m3fn or int8 [pages, kv_heads, page_size, head_dim] on a CUDA "
                             f"device and 3-dimensional scales, got {k.dtype} {tuple(k.shape)} on {k.device}")
        pages, kv_heads, page_size, head_dim = k.shape
        blocks = k_scale.shape[2]
        if blocks < 1 or page_size % blocks:
            raise ValueError(f"k_scale: {blocks} blocks in a page of {page_size} tokens")
        _check_sizes(pages, kv_heads, page_size, head_dim, page_size // blocks)
        _flat(k, "k", k.shape, k.dtype, k.device)
        _flat(v, "v", k.shape, k.dtype, k.device)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _flat(t, name, (pages, kv_heads, blocks), torch.float32, k.device)
        for t, name in ((k, "k"), (v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.data_ptr() & 15:
                raise ValueError(f"{name}: expected a 16-byte aligned tensor")
        self._tensors = k, v, k_scale, v_scale  # whose addresses _c holds
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, kv_heads, page_size, head_dim
        self.block, self.dtype, self.device = page_size // blocks, k.dtype, k.device
        self._c = _Cache(pages, kv_heads, page_size, self.block, head_dim, CACHE_TYPES[k.dtype],
                         *(t.data_ptr() for t in (k, v, k_scale, v_scale)))

    k = property(lambda self: self._tensors[0], doc="codes of the keys")
    v = property(lambda self: self._tensors[1], doc="codes of the values")
    k_scale = property(lambda self: self._tensors[2], doc="scales of the keys")
    v_scale = property(lambda self: self._tensors[3], doc="scales of the values")

    def _table(self, page_table, batch):
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table: expected int32 [batch, table_pages]")
        return _flat(page_table, "page_table", (batch, page_table.shape[1]), torch.int32, self.device)

    def _move(self, call, k, v, page_table, start, count, flags):
        batch, _, rows, _ = k.shape
        self._table(page_table, batch)
        _flat(start, "start", (batch,), torch.int32, self.device)
        _flat(count, "count", (batch,), torch.int32, self.device)
        if start is None:
            raise ValueError("start: expected int32 [batch]")
        if batch and rows:
            st = getattr(lib(), call)(ctypes.byref(self._c), batch, rows, _rows(k), _rows(v), IO_TYPES[k.dtype],
                                      _at(page_table), page_table.shape[1], _at(start), _at(count),
                                      _current_stream(self.device), flags)
            _check(st, call)

    def write(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor,
              count: Optional[torch.Tensor] = None, stream=None, check: bool = False):
        """Append rows to the cache: row i of k, v (bf16 or fp16 [batch,
        kv_heads, rows, d]) becomes token start[b] + i of sequence b, for i
        below count[b] (default: all rows).  start and count: int32 [batch] on
        the cache's device.  A block that gets rows takes the larger of its
        earlier tokens' scale and the one its new rows need; where the scale
        grows, the earlier tokens' codes are rounded again."""
        if not isinstance(k, torch.Tensor) or k.dtype not in IO_TYPES or k.dim() != 4:
            raise ValueError("k: expected bfloat16 or float16 [batch, kv_heads, rows, head_dim]")
        shape = (k.shape[0], self.kv_heads, k.shape[2], self.head_dim)
        with _on(self.device, stream):
            k = _input(k, "k", shape, k.dtype, self.device)
            v = _input(v, "v", shape, k.dtype, self.device)
            self._move("sta_cache_write", k, v, page_table, start, count, STA_CALL_CHECK if check else 0)

    def read(self, page_table: torch.Tensor, start: torch.Tensor, count: Optional[torch.Tensor], rows: int,
             dtype: torch.dtype = torch.bfloat16, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
             stream=None, check: bool = False):
        """(k, v) [batch, kv_heads, rows, d] with the values of tokens start[b],
        start[b] + 1, ... of sequence b, count[b] of them (None: all rows).
        Rows past count[b] or of absent pages are left as they were in a k or v
        that is passed in, and 0 in a new one."""
        if dtype not in IO_TYPES:
            raise ValueError(f"dtype: expected bfloat16 or float16, got {dtype}")
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table: expected int32 [batch, table_pages]")
        shape = (page_table.shape[0], self.kv_heads, int(rows), self.head_dim)
        with _on(self.device, stream):
            flags = STA_CALL_CHECK if check else 0
            if k is None and v is None:
                flags |= STA_READ_ZERO
                _, h, n, d = shape
                k, v = (torch.empty_strided(shape, (h * n * d, n * d, d, 1), dtype=dtype, device=self.device)
                        for _ in range(2))
            else:
                k, v = (torch.zeros(shape, dtype=dtype, device=self.device) if t is None
                        else _output(t, name, shape, dtype, self.device) for t, name in ((k, "k"), (v, "v")))
            self._move("sta_cache_read", k, v, page_table, start, count, flags)
        return k, v

    def attention(self, q: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor, window: int = 0,
                  sinks: int = 0, scale: float = 0.0, o: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, stream=None, check: bool = False, want_lse: bool = True):
        """(o, lse) of the last Nq positions of each sequence over its cached
        tokens: q [batch, heads, Nq, d], lengths int32 [batch] tokens in the
        cache, the queries' own among them.  The visible keys are those of
        window_forward with Nk = lengths[b].  Not differentiable: o carries no
        gradient of a q that requires one."""
        if not isinstance(q, torch.Tensor) or q.dtype not in IO_TYPES or q.dim() != 4:
            raise ValueError("q: expected bfloat16 or float16 [batch, heads, rows, head_dim]")
        batch, heads, nq, _ = q.shape
        shape = (batch, heads, nq, self.head_dim)
        with _on(self.device, stream):
            q = _input(q, "q", shape, q.dtype, self.device)
            self._table(page_table, batch)
            _flat(lengths, "lengths", (batch,), torch.int32, self.device)
            if lengths is None:
                raise ValueError("lengths: expected int32 [batch]")
            if o is None:
                o = _new(q)
            else:
                _output(o, "o", shape, q.dtype, self.device)
            if lse is None and want_lse:
                lse = _statistics(shape[:3], self.device)
            else:
                _flat(lse, "lse", shape[:3], torch.float32, self.device)
            if batch and nq:
                st = lib().sta_cache_attention(ctypes.byref(self._c), batch, heads, nq,
                                               _int32(window, "window"), _int32(sinks, "sinks"),
                                               float(scale), IO_TYPES[q.dtype], _rows(q), _rows(o), _at(lse),
                                               _at(page_table), page_table.shape[1], _at(lengths),
                                               _current_stream(self.device),
                                               STA_CALL_CHECK if check else 0)
                _check(st, "sta_cache_attention")
        return o, lse
