"""The paged 8-bit key/value cache of a hybrid's softmax-attention layers.

``Kv8Cache`` is a handle on the caller's cache tensors with the three device
operators of ``include/gdnspec.h``: ``attend`` (a transaction's rows over the
committed cache and themselves), ``append`` (commit of the accepted rows) and
``copy_pages``.  ``PagedKv`` owns such tensors together with the host page
tables: requests are opened, reserved, forked, freed and compacted there, and
one upload a transaction gives the kernels their tables.

All device work is asynchronous on the caller's stream; errors only the device
can see set bits in ``status`` (see the header).
"""
from __future__ import annotations

import ctypes
import math
from contextlib import nullcontext
from typing import Optional, Sequence, Tuple

import numpy as np
import torch

from . import binding as gs

PAGE_TOKENS = (16, 32, 64, 128)
HEAD_SIZES = (64, 128, 256)


# The current stream's handle without building a Stream object (a few microseconds a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream_object(stream):
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))


class Kv8Cache:
    """A handle on cache tensors the caller owns.

    kv:     uint8 (or float8_e4m3fn) [pages, layers, 2, h_kv, page_tokens, d]; a page of a layer contiguous
    scale:  fp32 [pages, layers, h_kv, 2]; a page of a layer contiguous
    status: int32 [1], the transaction's device status word
    """

    def __init__(self, kv: torch.Tensor, scale: torch.Tensor, h_q: int, status: torch.Tensor, window: int = 0,
                 sm_scale: Optional[float] = None):
        if kv.dim() != 6 or kv.shape[2] != 2 or kv.element_size() != 1:
            raise ValueError("kv must be 8-bit [pages, layers, 2, h_kv, page_tokens, d]")
        pages, layers, _, h_kv, page_tokens, d = kv.shape
        if kv.stride()[2:] != (h_kv * page_tokens * d, page_tokens * d, d, 1):
            raise ValueError("a page of a layer must be contiguous")
        if scale.shape != (pages, layers, h_kv, 2) or scale.dtype != torch.float32 or scale.stride()[2:] != (2, 1):
            raise ValueError("scale must be fp32 [pages, layers, h_kv, 2], a page of a layer contiguous")
        if status.dtype != torch.int32 or status.numel() != 1:
            raise ValueError("status must be one int32")
        if scale.device != kv.device or status.device != kv.device:
            raise ValueError("kv, scale and status must be on one device")
        self.kv, self.scale, self.status = kv, scale, status
        self.h_q, self.h_kv, self.d, self.page_tokens = h_q, h_kv, d, page_tokens
        self.c = gs.kv8_cache(h_q, h_kv, d, page_tokens, window, pages, layers,
                              1.0 / math.sqrt(d) if sm_scale is None else sm_scale, kv.data_ptr(), kv.stride(0),
                              kv.stride(1), scale.data_ptr(), scale.stride(0), scale.stride(1))
        self._c = ctypes.byref(self.c)
        self._device = kv.device
        self._index = kv.get_device()
        self._status = status.data_ptr()
        self._workspace = {}  # (B, max_len, max_rows, split_tokens) -> bytes

    def _rows(self, x: torch.Tensor, heads: int, name: str):
        """-> (address, row stride) of packed rows of heads."""
        shape, stride = x.shape, x.stride()
        if (x.dtype is not torch.bfloat16 or len(shape) != 3 or shape[1] != heads or shape[2] != self.d
                or stride[1] != self.d or stride[2] != 1 or x.get_device() != self._index):
            raise ValueError("%s must be bf16 [rows, %d, %d] with contiguous heads, on the cache's device"
                             % (name, heads, self.d))
        return x.data_ptr(), stride[0]

    def _ints(self, x: torch.Tensor, n: int, name: str):
        """-> address of a contiguous int32 list of at least n."""
        if (x.dtype is not torch.int32 or x.dim() != 1 or x.numel() < n or not x.is_contiguous()
                or x.get_device() != self._index):
            raise ValueError("%s must be a contiguous int32 list of at least %d, on the cache's device" % (name, n))
        return x.data_ptr()

    def _table(self, table: torch.Tensor, B: int):
        """-> (address, entries a row, row stride) of the page table."""
        shape, stride = table.shape, table.stride()
        if (table.dtype is not torch.int32 or len(shape) != 2 or shape[0] < B or (stride[1] != 1 and shape[1] > 1)
                or table.get_device() != self._index):
            raise ValueError("table must be int32 [requests, pages] with contiguous rows, on the cache's device")
        return table.data_ptr(), shape[1], stride[0]

    def attend(self, layer: int, table: torch.Tensor, cache_len: torch.Tensor, cu_rows: torch.Tensor,
               q: torch.Tensor, k_new: Optional[torch.Tensor], v_new: Optional[torch.Tensor], max_len: int,
               max_rows: int = gs.MAX_ROWS, split_tokens: int = 0, want_lse: bool = False,
               out: Optional[torch.Tensor] = None, stream=None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """-> (o bf16 [rows, h_q, d], lse fp32 [rows, h_q] or None); ``kv8_attend`` in the header.

        max_len and max_rows are host bounds on cache_len and on a request's rows."""
        B, R = cache_len.shape[0], q.shape[0]
        len_p, cu_p = self._ints(cache_len, B, "cache_len"), self._ints(cu_rows, B + 1, "cu_rows")
        table_p, table_n, table_s = self._table(table, B)
        q_p, q_s = self._rows(q, self.h_q, "q")
        k_p = k_s = v_p = v_s = 0
        if k_new is not None or v_new is not None:
            if k_new is None or v_new is None or k_new.shape[0] < R or v_new.shape[0] < R:
                raise ValueError("k_new and v_new come together and need a row for each of q's")
            k_p, k_s = self._rows(k_new, self.h_kv, "k_new")
            v_p, v_s = self._rows(v_new, self.h_kv, "v_new")
        key = (B, max_len, max_rows, split_tokens)
        need = self._workspace.get(key)
        if need is None:
            if len(self._workspace) > 4096:
                self._workspace.clear()
            need = self._workspace[key] = gs.lib.kv8_attend_workspace_bytes(self._c, *key)
        if stream is not None:
            # what the call allocates belongs to the stream it runs on
            stream = _stream_object(stream)
            before = torch.cuda.current_stream(self._device)
            torch.cuda.set_stream(stream)
        try:
            raw = _raw_stream(self._index)
            if out is None:
                out = torch.empty((R, self.h_q, self.d), dtype=torch.bfloat16, device=self._device)
                o_p, o_s = out.data_ptr(), self.h_q * self.d
            elif out.shape[0] < R:
                raise ValueError("out needs a row for each of q's")
            else:
                o_p, o_s = self._rows(out, self.h_q, "out")
            lse = torch.empty((R, self.h_q), dtype=torch.float32, device=self._device) if want_lse else None
            ws = torch.empty((need,), dtype=torch.uint8, device=self._device) if need else None
        finally:
            if stream is not None:
                torch.cuda.set_stream(before)
        st = gs.lib.kv8_attend(self._c, layer, B, R, cu_p, len_p, table_p, table_n, table_s, q_p, q_s, k_p or None, k_s,
                               v_p or None, v_s, o_p, o_s, lse.data_ptr() if want_lse else None, max_len, max_rows,
                               split_tokens, ws.data_ptr() if need else None, need, self._status, raw)
        if st != gs.GDN_OK:
            raise gs.GdnError("kv8_attend", st)
        return out, lse

    def append(self, layer: int, table: torch.Tensor, cache_len: torch.Tensor, cu_rows: torch.Tensor,
               k_new: torch.Tensor, v_new: torch.Tensor, accept_len: Optional[torch.Tensor] = None,
               max_rows: int = gs.MAX_ROWS, stream=None):
        """Commits the first accept_len[r] + 1 rows of each request (all rows without accept_len);
        ``kv8_append`` in the header."""
        B = cache_len.shape[0]
        len_p, cu_p = self._ints(cache_len, B, "cache_len"), self._ints(cu_rows, B + 1, "cu_rows")
        table_p, table_n, table_s = self._table(table, B)
        k_p, k_s = self._rows(k_new, self.h_kv, "k_new")
        v_p, v_s = self._rows(v_new, self.h_kv, "v_new")
        acc_p = None if accept_len is None else self._ints(accept_len, B, "accept_len")
        st = gs.lib.kv8_append(self._c, layer, B, min(k_new.shape[0], v_new.shape[0]), cu_p, len_p, table_p, table_n,
                               table_s, k_p, k_s, v_p, v_s, acc_p, max_rows, self._status,
                               _raw_stream(self._index) if stream is None else gs._stream(stream))
        if st != gs.GDN_OK:
            raise gs.GdnError("kv8_append", st)

    def copy_pages(self, src: torch.Tensor, dst: torch.Tensor, stream=None):
        """Page dst[i] <- page src[i], every layer; ``kv8_copy_pages`` in the header."""
        n = src.shape[0]
        if dst.shape != src.shape:
            raise ValueError("src and dst must be lists of one length")
        st = gs.lib.kv8_copy_pages(self._c, n, self._ints(src, n, "src"), self._ints(dst, n, "dst"), self._status,
                                   _raw_stream(self._index) if stream is None else gs._stream(stream))
        if st != gs.GDN_OK:
            raise gs.GdnError("kv8_copy_pages", st)


class PagedKv(Kv8Cache):
    """Cache tensors, page pool and host page tables of up to max_batch requests.

    A decode transaction: ``reserve`` room for its rows, ``upload`` the tables, ``attend`` every layer,
    ``append`` every layer once the accept lengths are on the device, ``advance`` once they are on the host."""

    def __init__(self, num_layers: int, num_pages: int, max_batch: int, max_tokens: int, h_q: int, h_kv: int, d: int,
                 page_tokens: int = 64, window: int = 0, sm_scale: Optional[float] = None, device="cuda",
                 status: Optional[torch.Tensor] = None):
        if d not in HEAD_SIZES or page_tokens not in PAGE_TOKENS:
            raise ValueError("d must be one of %r and page_tokens one of %r" % (HEAD_SIZES, PAGE_TOKENS))
        dev = torch.device(device)
        kv = torch.zeros((num_pages, num_layers, 2, h_kv, page_tokens, d), dtype=torch.uint8, device=dev)
        scale = torch.zeros((num_pages, num_layers, h_kv, 2), dtype=torch.float32, device=dev)
        if status is None:
            status = torch.zeros((1,), dtype=torch.int32, device=dev)
        super().__init__(kv, scale, h_q, status, window, sm_scale)
        self.pool = gs.Pool(num_pages)
        cap = -(-max_tokens // page_tokens)
        self.max_tokens = max_tokens
        self.tables = np.full((max_batch, cap), -1, dtype=np.int32)
        self.n_pages = np.zeros(max_batch, dtype=np.int32)
        self.length = np.zeros(max_batch, dtype=np.int32)
        self.dev_table = torch.full((max_batch, cap), -1, dtype=torch.int32, device=dev)
        self.dev_len = torch.zeros((max_batch,), dtype=torch.int32, device=dev)
        self._stage = torch.empty((max_batch, cap + 1), dtype=torch.int32)
        if dev.type == "cuda":
            self._stage = self._stage.pin_memory()
        self._staged: Optional[torch.cuda.Event] = None

    @property
    def max_len(self) -> int:
        return int(self.length.max(initial=0))

    def reserve(self, requests: Sequence[int], n_new: Sequence[int], stream=None):
        """Pages for n_new[i] more tokens of requests[i]; shared pages they would write into are copied.
        All or nothing for each request; the copies are queued even when a later request finds no page."""
        pairs = []
        try:
            for r, n in zip(requests, n_new):
                self.n_pages[r], pair = gs.kv8_pages_reserve(self.pool, self.tables[r], int(self.n_pages[r]),
                                                             int(self.length[r]), int(n), self.page_tokens)
                if pair:
                    pairs.append(pair)
        finally:
            self._copy(pairs, stream)

    def fork(self, src: int, dst: int, length: Optional[int] = None, stream=None):
        """Request dst (empty) becomes a second holder of the first tokens of src."""
        n = int(self.length[src]) if length is None else int(length)
        if self.n_pages[dst] or n > self.length[src]:
            raise ValueError("fork needs an empty request and at most the source's length")
        self.n_pages[dst], pair = gs.kv8_pages_fork(self.pool, self.tables[src], int(self.n_pages[src]), n,
                                                    self.page_tokens, self.tables[dst])
        self.length[dst] = n
        self._copy([pair] if pair else [], stream)

    def free(self, r: int):
        gs.kv8_pages_free(self.pool, self.tables[r], int(self.n_pages[r]))
        self.n_pages[r] = self.length[r] = 0

    def compact(self, stream=None) -> int:
        """Moves the live pages to the low end of the pool; -> pages moved."""
        src, dst = gs.kv8_pages_compact(self.pool, self.tables, self.n_pages)
        self._copy(list(zip(src.tolist(), dst.tolist())), stream)
        return len(src)

    def advance(self, requests: Sequence[int], n_new: Sequence[int]):
        """The committed tokens of a transaction become part of the requests."""
        for r, n in zip(requests, n_new):
            if int(self.length[r]) + int(n) > int(self.n_pages[r]) * self.page_tokens or n < 0:
                raise ValueError("request %d has no pages for %d more tokens" % (r, n))
        for r, n in zip(requests, n_new):
            self.length[r] += int(n)

    def upload(self, requests: Sequence[int], stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """-> (table [B, pages], cache_len [B]) on the device, row i for requests[i].  They are the same
        tensors every time: work that reads one upload's goes to the stream of the next, or is waited for first."""
        B, cap = len(requests), self.tables.shape[1]
        if self._staged is not None:
            self._staged.synchronize()  # the last upload has left the staging rows
        idx = np.asarray(requests, dtype=np.int64)
        stage = self._stage[:B].numpy()
        stage[:, :cap] = self.tables[idx]
        stage[:, cap] = self.length[idx]
        s = torch.cuda.current_stream() if stream is None else _stream_object(stream)
        with torch.cuda.stream(s):
            both = self._stage[:B].to(self.dev_table.device, non_blocking=True)
            self.dev_table[:B].copy_(both[:, :cap])
            self.dev_len[:B].copy_(both[:, cap])
            self._staged = torch.cuda.Event()
            self._staged.record()
        return self.dev_table[:B], self.dev_len[:B]

    def _copy(self, pairs, stream):
        if not pairs:
            return
        with nullcontext() if stream is None else torch.cuda.stream(_stream_object(stream)):
            ids = torch.tensor(pairs, dtype=torch.int32).t().contiguous().to(self.kv.device)
            self.copy_pages(ids[0], ids[1])
