"""What the paged 8-bit cache's calls refuse on the host, before anything is
launched (no GPU: no pointer here is ever followed)."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def gs():
    from speculative_decoding_hybrid_gb300 import build
    build.build()
    from speculative_decoding_hybrid_gb300 import binding
    return binding


def cache(gs, **kw):
    d = dict(h_q=8, h_kv=2, d=128, page_tokens=64, window=0, num_pages=10, num_layers=2, sm_scale=0.1, kv=4096,
             page_stride=2 * 32768, layer_stride=32768, scale=4096, scale_page_stride=8, scale_layer_stride=4)
    d.update(kw)
    c = gs.kv8_cache()
    for k, v in d.items():
        setattr(c, k, v)
    return c


def attend(gs, c, **kw):
    a = dict(layer=0, B=1, cap=4, cu=64, lens=64, table=64, pages=4, stride=4, q=64, qs=1024, k=64, ks=256, v=64,
             vs=256, o=64, os=1024, max_len=256, max_rows=4, split=0, ws=None, ws_n=0)
    a.update(kw)
    return gs.lib.kv8_attend(ctypes.byref(c) if c is not None else None, a["layer"], a["B"], a["cap"], a["cu"],
                             a["lens"], a["table"], a["pages"], a["stride"], a["q"], a["qs"], a["k"], a["ks"], a["v"],
                             a["vs"], a["o"], a["os"], None, a["max_len"], a["max_rows"], a["split"], a["ws"],
                             a["ws_n"], None, None)


def append(gs, c, **kw):
    a = dict(layer=0, B=1, cap=4, cu=64, lens=64, table=64, pages=4, stride=4, k=64, ks=256, v=64, vs=256, rows=4)
    a.update(kw)
    return gs.lib.kv8_append(ctypes.byref(c), a["layer"], a["B"], a["cap"], a["cu"], a["lens"], a["table"],
                             a["pages"], a["stride"], a["k"], a["ks"], a["v"], a["vs"], None, a["rows"], None, None)


def test_cache_shapes(gs):
    for kw, code in ((dict(d=96), gs.GDN_ERR_SHAPE), (dict(d=32), gs.GDN_ERR_SHAPE),
                     (dict(page_tokens=48), gs.GDN_ERR_SHAPE), (dict(page_tokens=256), gs.GDN_ERR_SHAPE),
                     (dict(h_q=7), gs.GDN_ERR_SHAPE), (dict(h_kv=0), gs.GDN_ERR_SHAPE),
                     (dict(h_q=130, h_kv=2), gs.GDN_ERR_SHAPE), (dict(window=-1), gs.GDN_ERR_ARG),
                     (dict(num_pages=0), gs.GDN_ERR_ARG), (dict(sm_scale=float("nan")), gs.GDN_ERR_ARG),
                     (dict(kv=None), gs.GDN_ERR_NULL), (dict(scale=None), gs.GDN_ERR_NULL),
                     (dict(page_stride=100), gs.GDN_ERR_ARG), (dict(page_stride=2 * 32768 + 8), gs.GDN_ERR_ARG),
                     (dict(layer_stride=16384), gs.GDN_ERR_ARG), (dict(kv=4100), gs.GDN_ERR_ARG),
                     (dict(scale_page_stride=3), gs.GDN_ERR_ARG), (dict(scale=4100), gs.GDN_ERR_ARG)):
        c = cache(gs, **kw)
        assert attend(gs, c) == code, kw
        assert append(gs, c) == code, kw
        assert gs.lib.kv8_copy_pages(ctypes.byref(c), 1, 64, 64, None, None) == code, kw
        assert gs.kv8_attend_workspace_bytes(c, 8, 1 << 20, 4) == 0
    assert attend(gs, None) == gs.GDN_ERR_NULL


def test_attend_arguments(gs):
    c = cache(gs)
    for kw, code in ((dict(layer=2), gs.GDN_ERR_ARG), (dict(layer=-1), gs.GDN_ERR_ARG), (dict(B=-1), gs.GDN_ERR_ARG),
                     (dict(B=65536), gs.GDN_ERR_ARG), (dict(cap=-1), gs.GDN_ERR_ARG), (dict(pages=-1), gs.GDN_ERR_ARG),
                     (dict(stride=-4), gs.GDN_ERR_ARG), (dict(max_len=-1), gs.GDN_ERR_ARG),
                     (dict(max_rows=17), gs.GDN_ERR_ARG), (dict(split=-1), gs.GDN_ERR_ARG),
                     (dict(cu=None), gs.GDN_ERR_NULL), (dict(lens=None), gs.GDN_ERR_NULL),
                     (dict(table=None), gs.GDN_ERR_NULL), (dict(q=None), gs.GDN_ERR_NULL),
                     (dict(o=None), gs.GDN_ERR_NULL), (dict(k=None), gs.GDN_ERR_NULL), (dict(v=None), gs.GDN_ERR_NULL),
                     (dict(q=72), gs.GDN_ERR_ARG), (dict(qs=1020), gs.GDN_ERR_ARG), (dict(qs=1000), gs.GDN_ERR_ARG),
                     (dict(ks=248), gs.GDN_ERR_ARG), (dict(v=66), gs.GDN_ERR_ARG), (dict(os=1 << 27), gs.GDN_ERR_ARG),
                     (dict(max_len=100000, pages=2000), gs.GDN_ERR_WORKSPACE)):
        assert attend(gs, c, **kw) == code, kw
    assert attend(gs, c, B=0) == gs.GDN_OK and attend(gs, c, max_rows=0) == gs.GDN_OK
    for bad in (0, 1_000_000_001):
        assert gs.lib.kv8_selftest_attend_timeout(ctypes.byref(c), 0, 1, 4, 64, 64, 64, 4, 4, 64, 1024, 64, 1024, 256,
                                                  4, 0, None, 0, None, bad, None) == gs.GDN_ERR_ARG


def test_append_and_copy_arguments(gs):
    c = cache(gs)
    for kw, code in ((dict(layer=2), gs.GDN_ERR_ARG), (dict(B=-1), gs.GDN_ERR_ARG), (dict(B=65536), gs.GDN_ERR_ARG),
                     (dict(rows=-1), gs.GDN_ERR_ARG), (dict(pages=1 << 30), gs.GDN_ERR_ARG),
                     (dict(B=2, stride=3), gs.GDN_ERR_ARG), (dict(k=None), gs.GDN_ERR_NULL),
                     (dict(v=None), gs.GDN_ERR_NULL), (dict(cu=None), gs.GDN_ERR_NULL),
                     (dict(table=None), gs.GDN_ERR_NULL), (dict(k=72), gs.GDN_ERR_ARG), (dict(ks=252), gs.GDN_ERR_ARG),
                     (dict(vs=128), gs.GDN_ERR_ARG)):
        assert append(gs, c, **kw) == code, kw
    assert append(gs, c, B=0) == gs.GDN_OK and append(gs, c, rows=0) == gs.GDN_OK
    copy = lambda n, s, t: gs.lib.kv8_copy_pages(ctypes.byref(c), n, s, t, None, None)
    assert copy(-1, 64, 64) == gs.GDN_ERR_ARG and copy(0, None, None) == gs.GDN_OK
    assert copy(1, None, 64) == gs.GDN_ERR_NULL and copy(1, 64, None) == gs.GDN_ERR_NULL


def test_workspace_goes_by_the_work(gs):
    """None for units that are not cut; with free cuts two parts a CTA whatever the batch; with given cuts one a piece."""
    c = cache(gs)
    ws = lambda *a: gs.kv8_attend_workspace_bytes(c, *a)
    assert ws(4, 0, 4) == 0 and ws(64, 1024, 4) == 0
    assert 0 < ws(1, 100000, 4) <= ws(64, 100000, 4) == ws(4096, 1 << 20, 4)
    assert ws(64, 100000, 4, 1 << 20) == 0
    assert ws(8, 128 * 10, 4, 128) == 8 * 2 * 10 * 16 * (128 * 4 + 8)
    assert ws(8, -1, 4) == 0 and ws(8, 1000, 17) == 0 and ws(8, 1000, 4, -1) == 0


def test_host_tables_refuse_null(gs):
    p = ctypes.byref(gs.Pool(4).c)
    t = np.zeros(4, np.int32)
    n = ctypes.c_int32(0)
    r = ctypes.byref(n)
    L = gs.lib
    assert L.kv8_pages_reserve(None, t.ctypes.data, 4, r, 0, 1, 16, r, r, r) == gs.GDN_ERR_NULL
    assert L.kv8_pages_reserve(p, None, 4, r, 0, 1, 16, r, r, r) == gs.GDN_ERR_NULL
    assert L.kv8_pages_fork(p, None, 1, 1, 16, t.ctypes.data, 4, r, r, r, r) == gs.GDN_ERR_NULL
    assert L.kv8_pages_free(None, t.ctypes.data, r) == gs.GDN_ERR_NULL
    assert L.kv8_pages_compact(p, 1, None, 4, t.ctypes.data, t.ctypes.data, t.ctypes.data, r) == gs.GDN_ERR_NULL
    assert L.kv8_pages_compact(p, -1, None, 4, None, t.ctypes.data, t.ctypes.data, r) == gs.GDN_ERR_ARG


def test_python_side_checks_without_a_gpu(gs):
    import torch

    from speculative_decoding_hybrid_gb300.kvcache import Kv8Cache, PagedKv
    kv = torch.zeros((6, 2, 2, 2, 32, 64), dtype=torch.uint8)
    sc = torch.zeros((6, 2, 2, 2))
    st = torch.zeros(1, dtype=torch.int32)
    Kv8Cache(kv, sc, 4, st)
    for bad in ((kv[:, :, :, :, :16], sc, 4, st), (kv.float(), sc, 4, st), (kv, sc[:5], 4, st),
                (kv, sc.double(), 4, st), (kv, sc, 4, st.long()), (kv[:, :, 0], sc, 4, st)):
        with pytest.raises(ValueError):
            Kv8Cache(*bad)
    with pytest.raises(ValueError):
        PagedKv(1, 4, 1, 64, 4, 2, 96, device="cpu")
    p = PagedKv(2, 8, 3, 128, 4, 2, 64, page_tokens=16, device="cpu")
    p.reserve([0], [20])
    with pytest.raises(ValueError):
        p.advance([0], [40])                      # more than was reserved
    p.advance([0], [20])
    with pytest.raises(ValueError):
        p.fork(0, 1, 21)                          # more than there is
    with pytest.raises(gs.GdnError):
        p.reserve([0], [200])                     # past max_tokens
    p.free(0)
    assert p.pool.free_list() and p.max_len == 0
