"""The attention layers' prompt side: rotary positions and attention over whole prompts.

What a prefill transaction does in a hybrid's softmax-attention layers, beside
``gdn_chunked_prefill`` in its GatedDeltaNet layers: ``Rope.rotate`` turns the
queries and new keys, ``attend_prompts`` computes the outputs of prompts without
earlier tokens (``Kv8Cache.attend_chunk`` those of rows behind a cache), and
``Kv8Cache.append`` commits the keys and values.

All device work is asynchronous on the caller's stream; errors only the device
can see set bits in ``status`` (see ``include/gdnspec.h``).
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import numpy as np
import torch

from . import binding as gs
from .kvcache import _BF16, _I32, _current_device, _raw_stream, _stream_on

SCALINGS = ("none", "linear", "base", "parts")


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, trained: int = 0,
                     slow: float = 1.0, fast: float = 32.0) -> Tuple[np.ndarray, float]:
    """-> (fp64 [rot/2] angular frequencies, the factor on cosine and sine).

    f_j = base^(-2j/rot), and for contexts `factor` times as long as the trained one:
    linear: every frequency over factor;
    base:   base * factor^(rot/(rot-2)), which leaves the fastest and divides the slowest by factor;
    parts:  frequencies that turn at least `fast` times in `trained` positions stay, those that turn at most `slow`
            times are divided by factor, in between a straight line in the number of turns; cosine and sine times
            1 + 0.1 ln(factor).  (A model trained with a line in the channel's number instead, with whole channels as
            its ends, or without the factor on cosine and sine, wants its own frequencies and magnitude.)"""
    if rot <= 0 or rot % 2:
        raise ValueError("rot is a positive even number of channels")
    if scaling not in SCALINGS:
        raise ValueError("scaling is one of %r" % (SCALINGS,))
    if not (base > 1.0 and math.isfinite(base) and factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("base is above 1 and factor at least 1")
    if scaling == "base":
        if rot < 4:
            raise ValueError("a scaled base wants rot of 4 or more")
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot)
    magnitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if trained <= 0 or not slow < fast:
            raise ValueError("scaling by parts wants the trained length and slow < fast")
        keep = np.clip((trained * f / (2.0 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        magnitude = 1.0 + 0.1 * math.log(factor)
    return f, magnitude


class Rope:
    """Rotary positions of d-channel heads: the first `rot` channels (default all) turn, in pairs (j, j + rot/2) or,
    interleaved, (2j, 2j + 1).  The frequencies are rope_frequencies(...) or given (`frequencies`, and with them
    `magnitude`, on cosine and sine)."""

    def __init__(self, d: int, rot: Optional[int] = None, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, trained: int = 0, device="cuda",
                 frequencies=None, magnitude: float = 1.0, slow: float = 1.0, fast: float = 32.0):
        rot = d if rot is None else rot
        if d <= 0 or d % 8 or d > 512 or rot <= 0 or rot % 2 or rot > d:
            raise ValueError("d is a multiple of 8 up to 512, rot an even number up to d")
        if frequencies is None:
            f, magnitude = rope_frequencies(rot, base, scaling, factor, trained, slow, fast)
        else:
            f = np.asarray(frequencies, dtype=np.float64)
            if f.shape != (rot // 2,) or not np.isfinite(f).all():
                raise ValueError("frequencies are rot/2 finite numbers")
        self.d, self.rot, self.interleaved, self.frequencies, self.magnitude = d, rot, bool(interleaved), f, magnitude
        turns = np.array([int(round(math.ldexp(x, 64))) % (1 << 64) for x in (f / (2.0 * math.pi)).tolist()],
                         dtype=np.uint64)
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        self._device = self.turns.device
        self._index = self.turns.get_device()
        self._turns = self.turns.data_ptr()
        self._spec = {}  # (h_q, h_kv) -> rope_spec

    def _bad(self, name: str):
        return ValueError("%s must be bf16 [rows, heads, %d] with contiguous heads on the table's device, a row for "
                          "each of the call's" % (name, self.d))

    def rotate(self, q: torch.Tensor, k: Optional[torch.Tensor], cu_rows: torch.Tensor,
               cache_len: Optional[torch.Tensor], status: torch.Tensor, in_place: bool = False,
               q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """-> (q, k) turned to positions cache_len[r] + i (``rope_rows`` in the header): new tensors, q_out and k_out,
        or in place.  k may be None."""
        # (the checks stand in the call: on few rows its time is its host side)
        d, index = self.d, self._index
        if index < 0:
            raise ValueError("the table must be on a GPU")
        B = cu_rows.numel() - 1
        if (cu_rows.dtype is not _I32 or B < 0 or not cu_rows.is_contiguous() or cu_rows.get_device() != index
                or status.dtype is not _I32 or status.numel() != 1 or status.get_device() != index):
            raise ValueError("cu_rows must be a contiguous int32 list and status one int32, on the table's device")
        len_p = None
        if cache_len is not None:
            if (cache_len.dtype is not _I32 or cache_len.numel() < B or not cache_len.is_contiguous()
                    or cache_len.get_device() != index):
                raise ValueError("cache_len must be a contiguous int32 list of the requests, on the table's device")
            len_p = cache_len.data_ptr()
        if in_place:
            if q_out is not None or k_out is not None:
                raise ValueError("in place there is no other output")
            q_out, k_out = q, k
        R, h_q, c = q.shape
        q_s, x, one = q.stride()
        if q.dtype is not _BF16 or c != d or one != 1 or (x != d and h_q > 1) or q.get_device() != index:
            raise self._bad("q")
        h_kv = k_s = 0
        if k is not None:
            n, h_kv, c = k.shape
            k_s, x, one = k.stride()
            if (k.dtype is not _BF16 or n != R or c != d or one != 1 or (x != d and h_kv > 1)
                    or k.get_device() != index):
                raise self._bad("k")
        elif k_out is not None:
            raise ValueError("k_out without k")
        if _current_device() != index:
            with torch.cuda.device(index):  # the library launches on the current one
                return self.rotate(q, k, cu_rows, cache_len, status, False, q_out, k_out, stream)
        if stream is not None:
            # what the call allocates belongs to the stream it runs on
            stream = _stream_on(stream, index)
            before = torch.cuda.current_stream(self._device)
            torch.cuda.set_stream(stream)
        try:
            raw = _raw_stream(index)
            if q_out is None:
                q_out, qo_s = torch.empty((R, h_q, d), dtype=_BF16, device=self._device), h_q * d
            else:
                n, h, c = q_out.shape
                qo_s, x, one = q_out.stride()
                if (q_out.dtype is not _BF16 or n != R or h != h_q or c != d or one != 1 or (x != d and h > 1)
                        or q_out.get_device() != index):
                    raise self._bad("q_out")
            ko_s = 0
            if k_out is not None:
                n, h, c = k_out.shape
                ko_s, x, one = k_out.stride()
                if (k_out.dtype is not _BF16 or n != R or h != h_kv or c != d or one != 1 or (x != d and h > 1)
                        or k_out.get_device() != index):
                    raise self._bad("k_out")
            elif k is not None:
                k_out, ko_s = torch.empty((R, h_kv, d), dtype=_BF16, device=self._device), h_kv * d
        finally:
            if stream is not None:
                torch.cuda.set_stream(before)
        if R <= 1:
            q_s = qo_s = h_q * d  # a single row's stride says nothing
            k_s = ko_s = h_kv * d
        spec = self._spec.get((h_q, h_kv))
        if spec is None:
            spec = self._spec[h_q, h_kv] = ctypes.byref(gs.rope_spec(h_q, h_kv, d, self.rot, int(self.interleaved),
                                                                     self.magnitude))
        st = gs.lib.rope_rows(spec, B, R, cu_rows.data_ptr(), len_p, self._turns, q.data_ptr(), q_s, q_out.data_ptr(),
                              qo_s, k.data_ptr() if h_kv else None, k_s, k_out.data_ptr() if h_kv else None, ko_s,
                              status.data_ptr(), raw)
        if st != gs.GDN_OK:
            raise gs.GdnError("rope_rows", st)
        return q_out, k_out


# A call's head layout and the workspace that its sizes want, by the arguments that fix them.
_workspace = {}


def _bad_rows(name: str, heads: int, d: int):
    return ValueError("%s must be bf16 [rows, %d, %d] with contiguous heads on q's device, a row for each of the "
                      "call's" % (name, heads, d))


def attend_prompts(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_rows: torch.Tensor, max_rows: int,
                   status: torch.Tensor, window: int = 0, sm_scale: Optional[float] = None, want_lse: bool = False,
                   out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """-> (o bf16 [rows, h_q, d], lse fp32 [rows, h_q] or None); ``attn_prompts`` in the header.

    q [rows, h_q, d], k and v [rows, h_kv, d]: packed prompts; max_rows is a host bound on a prompt's rows."""
    R, h_q, d = q.shape
    q_s, x, one = q.stride()
    index = q.get_device()
    if index < 0:
        raise ValueError("the rows must be on a GPU")
    B = cu_rows.numel() - 1
    if (cu_rows.dtype is not _I32 or B < 0 or not cu_rows.is_contiguous() or cu_rows.get_device() != index
            or status.dtype is not _I32 or status.numel() != 1 or status.get_device() != index):
        raise ValueError("cu_rows must be a contiguous int32 list and status one int32, on the rows' device")
    if q.dtype is not _BF16 or one != 1 or (x != d and h_q > 1):
        raise _bad_rows("q", h_q, d)
    n, h_kv, c = k.shape
    k_s, x, one = k.stride()
    if k.dtype is not _BF16 or n < R or c != d or one != 1 or (x != d and h_kv > 1) or k.get_device() != index:
        raise _bad_rows("k", h_kv, d)
    k1 = n <= 1
    n, h, c = v.shape
    v_s, x, one = v.stride()
    if (v.dtype is not _BF16 or n < R or h != h_kv or c != d or one != 1 or (x != d and h > 1)
            or v.get_device() != index):
        raise _bad_rows("v", h_kv, d)
    if n <= 1:
        v_s = h_kv * d  # a single row's stride says nothing
    if k1:
        k_s = h_kv * d
    if R <= 1:
        q_s = h_q * d
    o_s = h_q * d
    if out is not None:
        n, h, c = out.shape
        o_s, x, one = out.stride()
        if (out.dtype is not _BF16 or n < R or h != h_q or c != d or one != 1 or (x != d and h > 1)
                or out.get_device() != index):
            raise _bad_rows("out", h_q, d)
        if n <= 1:
            o_s = h_q * d
    if sm_scale is not None:
        sm_scale = float(sm_scale)  # (a tensor would be a key by its identity, not by its value)
    key = (h_q, h_kv, d, window, sm_scale, B, R, max_rows)
    plan = _workspace.get(key)
    if plan is None:
        if len(_workspace) > 4096:
            _workspace.clear()
        dims = gs.attn_dims(h_q, h_kv, d, window, 1.0 / math.sqrt(d) if sm_scale is None else sm_scale)
        plan = _workspace[key] = ctypes.byref(dims), gs.attn_prompts_workspace_bytes(dims, B, R, max_rows)
    dims, need = plan
    device = q.device
    if _current_device() != index:
        with torch.cuda.device(index):  # the library launches on the current one
            return attend_prompts(q, k, v, cu_rows, max_rows, status, window, sm_scale, want_lse, out, stream)
    if stream is not None:
        # what the call allocates belongs to the stream it runs on
        stream = _stream_on(stream, index)
        before = torch.cuda.current_stream(device)
        torch.cuda.set_stream(stream)
    try:
        raw = _raw_stream(index)
        if out is None:
            out = torch.empty((R, h_q, d), dtype=_BF16, device=device)
        lse = torch.empty((R, h_q), dtype=torch.float32, device=device) if want_lse else None
        ws = torch.empty((need,), dtype=torch.uint8, device=device) if need else None
    finally:
        if stream is not None:
            torch.cuda.set_stream(before)
    st = gs.lib.attn_prompts(dims, B, R, cu_rows.data_ptr(), q.data_ptr(), q_s, k.data_ptr(), k_s, v.data_ptr(), v_s,
                             out.data_ptr(), o_s, lse.data_ptr() if want_lse else None, max_rows,
                             ws.data_ptr() if need else None, need, status.data_ptr(), raw)
    if st != gs.GDN_OK:
        raise gs.GdnError("attn_prompts", st)
    return out, lse
