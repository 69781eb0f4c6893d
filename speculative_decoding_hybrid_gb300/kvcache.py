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
_BF16, _I32 = torch.bfloat16, torch.int32


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

    # The checks stand in the calls themselves: on small transactions a call's time is
    # its host side, and a Python function a tensor cost 2.4 of 16 us.

    def _bad_rows(self, name: str, heads: int):
        return ValueError("%s must be bf16 [rows, %d, %d] with contiguous heads on the cache's device, a row for each "
                          "of the call's" % (name, heads, self.d))

    def _bad_lists(self, names: str):
        return ValueError("table must be int32 [requests, pages] with contiguous rows, and %s contiguous int32 lists "
                          "that fit it, on the cache's device" % names)

    def attend(self, layer: int, table: torch.Tensor, cache_len: torch.Tensor, cu_rows: torch.Tensor,
               q: torch.Tensor, k_new: Optional[torch.Tensor], v_new: Optional[torch.Tensor], max_len: int,
               max_rows: int = gs.MAX_ROWS, split_tokens: int = 0, want_lse: bool = False,
               out: Optional[torch.Tensor] = None, stream=None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """-> (o bf16 [rows, h_q, d], lse fp32 [rows, h_q] or None); ``kv8_attend`` in the header.

        max_len and max_rows are host bounds on cache_len and on a request's rows."""
        h_q, h_kv, d, device = self.h_q, self.h_kv, self.d, self._index
        B = cache_len.numel()
        tables, pages = table.shape
        table_s, one = table.stride()
        if (table.dtype is not _I32 or cache_len.dtype is not _I32 or cu_rows.dtype is not _I32 or tables < B
                or (one != 1 and pages > 1) or cu_rows.numel() <= B or not cache_len.is_contiguous()
                or not cu_rows.is_contiguous() or table.get_device() != device or cache_len.get_device() != device
                or cu_rows.get_device() != device):
            raise self._bad_lists("cache_len and cu_rows")
        R, a, b = q.shape
        q_s, c, one = q.stride()
        if (q.dtype is not _BF16 or a != h_q or b != d or (c != d and h_q > 1) or one != 1
                or q.get_device() != device):
            raise self._bad_rows("q", h_q)
        if R <= 1:
            q_s = h_q * d  # a single row's stride, as a single head's, says nothing
        k_p = v_p = None
        k_s = v_s = 0
        if k_new is not None or v_new is not None:
            if k_new is None or v_new is None:
                raise ValueError("k_new and v_new come together")
            n, a, b = k_new.shape
            k_s, c, one = k_new.stride()
            if (k_new.dtype is not _BF16 or n < R or a != h_kv or b != d or (c != d and h_kv > 1) or one != 1
                    or k_new.get_device() != device):
                raise self._bad_rows("k_new", h_kv)
            if n <= 1:
                k_s = h_kv * d
            n, a, b = v_new.shape
            v_s, c, one = v_new.stride()
            if (v_new.dtype is not _BF16 or n < R or a != h_kv or b != d or (c != d and h_kv > 1) or one != 1
                    or v_new.get_device() != device):
                raise self._bad_rows("v_new", h_kv)
            if n <= 1:
                v_s = h_kv * d
            k_p, v_p = k_new.data_ptr(), v_new.data_ptr()
        o_s = h_q * d
        if out is not None:
            n, a, b = out.shape
            o_s, c, one = out.stride()
            if (out.dtype is not _BF16 or n < R or a != h_q or b != d or (c != d and h_q > 1) or one != 1
                    or out.get_device() != device):
                raise self._bad_rows("out", h_q)
            if n <= 1:
                o_s = h_q * d
        key = (B, max_len, max_rows, split_tokens)
        need = self._workspace.get(key)
        if need is None:
            if len(self._workspace) > 4096:
                self._workspace.clear()
            need = self._workspace[key] = gs.lib.kv8_attend_workspace_bytes(self._c, *key)
        if stream is not None:
            # what the call allocates belongs to the stream it runs on
            before = torch.cuda.current_stream(self._device)
            torch.cuda.set_stream(_stream_object(stream))
        try:
            raw = _raw_stream(device)
            if out is None:
                out = torch.empty((R, h_q, d), dtype=_BF16, device=self._device)
            lse = torch.empty((R, h_q), dtype=torch.float32, device=self._device) if want_lse else None
            ws = torch.empty((need,), dtype=torch.uint8, device=self._device) if need else None
        finally:
            if stream is not None:
                torch.cuda.set_stream(before)
        st = gs.lib.kv8_attend(self._c, layer, B, R, cu_rows.data_ptr(), cache_len.data_ptr(), table.data_ptr(), pages,
                               table_s, q.data_ptr(), q_s, k_p, k_s, v_p, v_s, out.data_ptr(), o_s,
                               lse.data_ptr() if want_lse else None, max_len, max_rows, split_tokens,
                               ws.data_ptr() if need else None, need, self._status, raw)
        if st != gs.GDN_OK:
            raise gs.GdnError("kv8_attend", st)
        return out, lse

    def append(self, layer: int, table: torch.Tensor, cache_len: torch.Tensor, cu_rows: torch.Tensor,
               k_new: torch.Tensor, v_new: torch.Tensor, accept_len: Optional[torch.Tensor] = None,
               max_rows: int = gs.MAX_ROWS, stream=None):
        """Commits the first accept_len[r] + 1 rows of each request (all rows without accept_len);
        ``kv8_append`` in the header."""
        h_kv, d, device = self.h_kv, self.d, self._index
        B = cache_len.numel()
        tables, pages = table.shape
        table_s, one = table.stride()
        if (table.dtype is not _I32 or cache_len.dtype is not _I32 or cu_rows.dtype is not _I32 or tables < B
                or (one != 1 and pages > 1) or cu_rows.numel() <= B or not cache_len.is_contiguous()
                or not cu_rows.is_contiguous() or table.get_device() != device or cache_len.get_device() != device
                or cu_rows.get_device() != device):
            raise self._bad_lists("cache_len and cu_rows")
        acc_p = None
        if accept_len is not None:
            if (accept_len.dtype is not _I32 or accept_len.numel() < B or not accept_len.is_contiguous()
                    or accept_len.get_device() != device):
                raise self._bad_lists("accept_len")
            acc_p = accept_len.data_ptr()
        R, a, b = k_new.shape
        k_s, c, one = k_new.stride()
        if (k_new.dtype is not _BF16 or a != h_kv or b != d or (c != d and h_kv > 1) or one != 1
                or k_new.get_device() != device):
            raise self._bad_rows("k_new", h_kv)
        n, a, b = v_new.shape
        v_s, c, one = v_new.stride()
        if (v_new.dtype is not _BF16 or n != R or a != h_kv or b != d or (c != d and h_kv > 1) or one != 1
                or v_new.get_device() != device):
            raise self._bad_rows("v_new", h_kv)
        if R <= 1:
            k_s = v_s = h_kv * d
        st = gs.lib.kv8_append(self._c, layer, B, R, cu_rows.data_ptr(), cache_len.data_ptr(), table.data_ptr(), pages,
                               table_s, k_new.data_ptr(), k_s, v_new.data_ptr(), v_s, acc_p, max_rows, self._status,
                               _raw_stream(device) if stream is None else gs._stream(stream))
        if st != gs.GDN_OK:
            raise gs.GdnError("kv8_append", st)

    def copy_pages(self, src: torch.Tensor, dst: torch.Tensor, stream=None):
        """Page dst[i] <- page src[i], every layer; ``kv8_copy_pages`` in the header."""
        n = src.numel()
        if (src.dtype is not _I32 or dst.dtype is not _I32 or dst.numel() != n or not src.is_contiguous()
                or not dst.is_contiguous() or src.get_device() != self._index or dst.get_device() != self._index):
            raise ValueError("src and dst must be contiguous int32 lists of one length on the cache's device")
        st = gs.lib.kv8_copy_pages(self._c, n, src.data_ptr(), dst.data_ptr(), self._status,
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
        s = torch.cuda.current_stream(self._device) if stream is None else _stream_object(stream)
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
