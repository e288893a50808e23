"""Python face of libsgd's paged 8-bit cache: the target model's keys and values.

What the verification pass of a draft needs next to SuffixDrafter.verify: the
1 + num_valid new tokens of every row enter the cache (write) and attend over
it (attend).  Every method marshals pointers and sizes and calls one C entry
point of include/sgd.h.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib as L
from .drafter import _DTYPES, SuffixDrafter, _stream_handle

_F8 = torch.float8_e4m3fn


class KVCache:
    """A paged cache of keys and values, held as e4m3 with one power-of-two
    scale per page and head.

    k, v: float8_e4m3fn [num_layers, num_pages, kv_heads, page_size, head_dim];
    k_scale, v_scale: float32 [num_layers, num_pages, kv_heads]; a value is its
    byte times its scale.  `storage` gives these four tensors (in that order)
    instead of new ones.  Position j of row b is in page block_table[b, j //
    page_size], slot j % page_size, and pages are handed out by the caller.

    The tokens of a call are packed: row b's are q_start[b] .. q_start[b + 1],
    the last ones of its seq_lens[b] tokens.  For a verification pass these are
    the row's last token and its drafts; after it, seq_lens simply does not
    advance past a rejected draft and the next write overwrites it.  (A draft of
    much larger keys or values than its page's other tokens holds these at its
    scale, within 2^-10 of it, and they stay so rounded when it is rejected.)
    """

    def __init__(self, num_pages: int, page_size: int, kv_heads: int, head_dim: int, max_batch: int,
                 max_pages_per_row: int, q_heads: Optional[int] = None, num_layers: int = 1,
                 storage: Optional[Tuple[torch.Tensor, ...]] = None, device: int = 0):
        self._h = None
        self._lib = L.load()
        cfg = L.SgdKvConfig(num_pages, page_size, kv_heads, q_heads if q_heads is not None else kv_heads,
                            head_dim, max_batch, max_pages_per_row)
        self.cfg = cfg
        self.device = torch.device("cuda", device)
        self._index = device
        torch.cuda.init()
        with torch.cuda.device(self.device):
            torch.zeros(1, device=self.device)  # make the primary context current
            h = ctypes.c_void_p()
            self._check(self._lib.sgd_kv_create(ctypes.byref(cfg), device, ctypes.byref(h)), "sgd_kv_create")
        self._h = h
        shape = (num_layers, num_pages, kv_heads, page_size, head_dim)
        if storage is None:
            storage = (torch.zeros(shape, dtype=torch.uint8, device=self.device).view(_F8),
                       torch.zeros(shape, dtype=torch.uint8, device=self.device).view(_F8),
                       torch.ones(shape[:3], device=self.device), torch.ones(shape[:3], device=self.device))
        for t, want, dtype in zip(storage, (shape, shape, shape[:3], shape[:3]),
                                  (_F8, _F8, torch.float32, torch.float32)):
            if tuple(t.shape) != want or t.dtype != dtype or not t.is_contiguous() or t.device != self.device:
                raise ValueError("storage must be contiguous tensors on %s: two %s of %s, two %s of %s"
                                 % (self.device, _F8, shape, torch.float32, shape[:3]))
        self.k, self.v, self.k_scale, self.v_scale = storage
        self.kv_heads, self.q_heads, self.head_dim = kv_heads, cfg.q_heads, head_dim
        self.page_size, self.max_batch, self.max_pages = page_size, max_batch, max_pages_per_row
        self._layers = [L.SgdKvLayer(*(t[i].data_ptr() for t in storage)) for i in range(num_layers)]
        self._layer_refs = [ctypes.addressof(x) for x in self._layers]

    _check = staticmethod(SuffixDrafter._check)
    _t = SuffixDrafter._t

    def _new(self, t: torch.Tensor, heads: int, name: str):
        """A packed [N, heads, head_dim] tensor whose last dimension is contiguous."""
        if t.get_device() != self._index:
            raise ValueError("%s must be on %s" % (name, self.device))
        if t.dim() != 3 or t.shape[1:] != (heads, self.head_dim) or t.stride(2) != 1:
            raise ValueError("%s must be [N, %d, %d] with a contiguous last dimension"
                             % (name, heads, self.head_dim))
        return t.data_ptr()

    def _rows(self, block_table: torch.Tensor, lens: torch.Tensor, starts: torch.Tensor) -> int:
        B = lens.shape[0]
        if block_table.shape != (B, self.max_pages) or starts.shape[0] != B + 1:
            raise ValueError("block_table must be [B, %d], the lengths [B] and the starts [B + 1]"
                             % self.max_pages)
        return B

    def write(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
              q_start: torch.Tensor, layer: int = 0, stream=None) -> None:
        """Writes the packed new keys and values [N, kv_heads, head_dim]
        (float32, float16 or bfloat16; slices of one projection's output are
        taken as they are).  seq_lens [B] counts the new tokens."""
        B = self._rows(block_table, seq_lens, q_start)
        dtype = _DTYPES.get(k.dtype)
        if dtype is None or v.dtype is not k.dtype or v.shape != k.shape:
            raise ValueError("k and v must have one shape, and one type of float32, float16 or bfloat16")
        t = self._t
        kt, kh, _ = k.stride()
        vt, vh, _ = v.stride()
        st = self._lib.sgd_kv_write(
            self._h, self._layer_refs[layer], self._new(k, self.kv_heads, "k"), self._new(v, self.kv_heads, "v"),
            dtype, kt, kh, vt, vh, t(block_table, name="block_table"), t(seq_lens, name="seq_lens"),
            t(q_start, name="q_start"), B, k.shape[0], _stream_handle(stream, self._index))
        if st < 0:
            raise L.SgdError(st, "sgd_kv_write")

    def read(self, block_table: torch.Tensor, start: torch.Tensor, out_start: torch.Tensor,
             out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, total: Optional[int] = None,
             dtype: torch.dtype = torch.bfloat16, layer: int = 0,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Keys and values of positions start[b], start[b] + 1, ... of row b as
        rows out_start[b] .. out_start[b + 1] of two [total, kv_heads, head_dim]
        tensors; `out` gives them, else `total` and `dtype` do."""
        B = self._rows(block_table, start, out_start)
        if out is None:
            if total is None:
                raise ValueError("read needs out or total")
            out = tuple(torch.empty((total, self.kv_heads, self.head_dim), dtype=dtype, device=self.device)
                        for _ in range(2))
        k, v = out
        dtype = _DTYPES.get(k.dtype)
        if dtype is None or v.dtype is not k.dtype or v.shape != k.shape or not k.is_contiguous() \
                or not v.is_contiguous():
            raise ValueError("out must be two contiguous tensors of one shape and type")
        t = self._t
        st = self._lib.sgd_kv_read(
            self._h, self._layer_refs[layer], t(block_table, name="block_table"), t(start, name="start"),
            t(out_start, name="out_start"), B, k.shape[0], self._new(k, self.kv_heads, "out"),
            self._new(v, self.kv_heads, "out"), dtype, _stream_handle(stream, self._index))
        if st < 0:
            raise L.SgdError(st, "sgd_kv_read")
        return k, v

    def attend(self, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
               q_start: torch.Tensor, max_q: int, scale: Optional[float] = None, window: int = 0,
               sinks: int = 0, out: Optional[torch.Tensor] = None, layer: int = 0,
               stream=None) -> torch.Tensor:
        """Attention of the packed new tokens q [N, q_heads, head_dim] (float16
        or bfloat16), already written, over their rows' cache: a token sees the
        positions up to its own, with window > 0 only the last `window` of them
        and the first `sinks`.  max_q: the most new tokens of any row."""
        B = self._rows(block_table, seq_lens, q_start)
        dtype = _DTYPES.get(q.dtype)
        if dtype is None or dtype == L.F32:
            raise ValueError("q must be float16 or bfloat16")
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        elif out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        t, at = self._t, self._new(q, self.q_heads, "q")
        qt, qh, _ = q.stride()
        st = self._lib.sgd_kv_attend(
            self._h, self._layer_refs[layer], at, dtype, qt, qh, t(block_table, name="block_table"),
            t(seq_lens, name="seq_lens"), t(q_start, name="q_start"), B, q.shape[0], max_q,
            scale if scale is not None else self.head_dim ** -0.5, window, sinks, t(out, q.dtype, "out"),
            _stream_handle(stream, self._index))
        if st < 0:
            raise L.SgdError(st, "sgd_kv_attend")
        return out

    # -- diagnostics ----------------------------------------------------------
    def get_error(self, clear: bool = False) -> int:
        f = ctypes.c_uint32()
        self._check(self._lib.sgd_kv_get_error(self._h, ctypes.byref(f), int(bool(clear))),
                    "sgd_kv_get_error")
        return int(f.value)

    def memory(self) -> int:
        """Device bytes the handle allocated (the cache itself is not among them)."""
        n = ctypes.c_int64()
        self._check(self._lib.sgd_kv_memory(self._h, ctypes.byref(n)), "sgd_kv_memory")
        return int(n.value)

    def launch_count(self) -> int:
        c = ctypes.c_uint64()
        self._check(self._lib.sgd_kv_launch_count(self._h, ctypes.byref(c)), "sgd_kv_launch_count")
        return int(c.value)

    def close(self) -> None:
        if self._h:
            self._lib.sgd_kv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
