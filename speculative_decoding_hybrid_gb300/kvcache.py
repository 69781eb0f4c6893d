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


def _on(stream):
    """(context in which to allocate, raw handle) of a stream argument."""
    if stream is None:
        return nullcontext(), torch.cuda.current_stream().cuda_stream
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream), stream.cuda_stream


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
        self._q, self._kv = ((h_q, d), (d, 1)), ((h_kv, d), (d, 1))

    @staticmethod
    def _rows(x: torch.Tensor, want, name: str):
        if x.dtype != torch.bfloat16 or x.shape[1:] != want[0] or x.stride()[1:] != want[1]:
            raise ValueError("%s must be bf16 [rows, %d, %d] with contiguous heads" % (name, *want[0]))
        return x.data_ptr(), x.stride(0)

    @staticmethod
    def _tables(table, cache_len, cu_rows):
        if table.dim() != 2 or table.stride(1) != 1:
            raise ValueError("table must be int32 [requests, pages] with contiguous rows")
        if not (table.dtype == cache_len.dtype == cu_rows.dtype == torch.int32):
            raise ValueError("table, cache_len and cu_rows must be int32")
        B = cache_len.shape[0]
        if table.shape[0] < B or cu_rows.shape[0] < B + 1 or not (cache_len.is_contiguous()
                                                                  and cu_rows.is_contiguous()):
            raise ValueError("cache_len [B], cu_rows [B + 1] and table [B, pages] do not fit together")
        return B

    def attend(self, layer: int, table: torch.Tensor, cache_len: torch.Tensor, cu_rows: torch.Tensor,
               q: torch.Tensor, k_new: Optional[torch.Tensor], v_new: Optional[torch.Tensor], max_len: int,
               max_rows: int = gs.MAX_ROWS, split_tokens: int = 0, want_lse: bool = False,
               out: Optional[torch.Tensor] = None, stream=None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """-> (o bf16 [rows, h_q, d], lse fp32 [rows, h_q] or None); ``kv8_attend`` in the header.

        max_len and max_rows are host bounds on cache_len and on a request's rows."""
        B = self._tables(table, cache_len, cu_rows)
        qp, qs = self._rows(q, self._q, "q")
        kp = ks = vp = vs = 0
        R = q.shape[0]
        if k_new is not None:
            kp, ks = self._rows(k_new, self._kv, "k_new")
            vp, vs = self._rows(v_new, self._kv, "v_new")
            if k_new.shape[0] < R or v_new.shape[0] < R:
                raise ValueError("k_new and v_new need a row for each of q's")
        ctx, raw = _on(stream)
        need = gs.lib.kv8_attend_workspace_bytes(self._c, B, max_len, max_rows, split_tokens)
        with ctx:
            if out is None:
                out = torch.empty((R, self.h_q, self.d), dtype=torch.bfloat16, device=q.device)
            lse = torch.empty((R, self.h_q), dtype=torch.float32, device=q.device) if want_lse else None
            ws = torch.empty((need,), dtype=torch.uint8, device=q.device) if need else None
        op, os_ = self._rows(out, self._q, "out")
        if out.shape[0] < R:
            raise ValueError("out needs a row for each of q's")
        st = gs.lib.kv8_attend(self._c, layer, B, R, cu_rows.data_ptr(), cache_len.data_ptr(), table.data_ptr(),
                               table.shape[1] if B == 1 else table.stride(0), qp, qs, kp or None, ks, vp or None, vs,
                               op, os_, lse.data_ptr() if want_lse else None, max_len, max_rows, split_tokens,
                               ws.data_ptr() if need else None, need, self.status.data_ptr(), raw)
        if st != gs.GDN_OK:
            raise gs.GdnError("kv8_attend", st)
        return out, lse

    def append(self, layer: int, table: torch.Tensor, cache_len: torch.Tensor, cu_rows: torch.Tensor,
               k_new: torch.Tensor, v_new: torch.Tensor, accept_len: Optional[torch.Tensor] = None,
               max_rows: int = gs.MAX_ROWS, stream=None):
        """Commits the first accept_len[r] + 1 rows of each request (all rows without accept_len);
        ``kv8_append`` in the header."""
        B = self._tables(table, cache_len, cu_rows)
        kp, ks = self._rows(k_new, self._kv, "k_new")
        vp, vs = self._rows(v_new, self._kv, "v_new")
        if accept_len is not None and (accept_len.dtype != torch.int32 or accept_len.shape[0] < B
                                       or not accept_len.is_contiguous()):
            raise ValueError("accept_len must be int32 [requests]")
        raw = torch.cuda.current_stream().cuda_stream if stream is None else gs._stream(stream)
        st = gs.lib.kv8_append(self._c, layer, B, min(k_new.shape[0], v_new.shape[0]), cu_rows.data_ptr(),
                               cache_len.data_ptr(), table.data_ptr(),
                               table.shape[1] if B == 1 else table.stride(0), kp, ks, vp, vs,
                               None if accept_len is None else accept_len.data_ptr(), max_rows,
                               self.status.data_ptr(), raw)
        if st != gs.GDN_OK:
            raise gs.GdnError("kv8_append", st)

    def copy_pages(self, src: torch.Tensor, dst: torch.Tensor, stream=None):
        """Page dst[i] <- page src[i], every layer; ``kv8_copy_pages`` in the header."""
        if src.dtype != torch.int32 or dst.dtype != torch.int32 or src.shape != dst.shape or src.dim() != 1 \
                or not (src.is_contiguous() and dst.is_contiguous()):
            raise ValueError("src and dst must be int32 lists of one length")
        raw = torch.cuda.current_stream().cuda_stream if stream is None else gs._stream(stream)
        st = gs.lib.kv8_copy_pages(self._c, src.shape[0], src.data_ptr(), dst.data_ptr(), self.status.data_ptr(), raw)
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
        """-> (table [B, pages], cache_len [B]) on the device, row i for requests[i]."""
        B, cap = len(requests), self.tables.shape[1]
        if self._staged is not None:
            self._staged.synchronize()  # the last upload has left the staging rows
        idx = np.asarray(requests, dtype=np.int64)
        stage = self._stage[:B].numpy()
        stage[:, :cap] = self.tables[idx]
        stage[:, cap] = self.length[idx]
        s = torch.cuda.current_stream() if stream is None else stream
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
        ctx, _ = _on(stream)
        with ctx:
            ids = torch.tensor(pairs, dtype=torch.int32).t().contiguous().to(self.kv.device)
            self.copy_pages(ids[0], ids[1])
