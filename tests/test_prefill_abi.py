"""What the prompt side's calls refuse on the host, before anything is launched (no GPU: no pointer here is ever
followed), and the frequencies of rotary positions."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def gs():
    from speculative_decoding_hybrid_gb300 import build
    build.build()
    from speculative_decoding_hybrid_gb300 import binding
    return binding


def rope(gs, spec=None, **kw):
    a = dict(B=1, cap=4, cu=64, lens=64, turns=64, q=64, qs=1024, qo=4096, qos=1024, k=64, ks=256, ko=4096, kos=256)
    a.update(kw)
    s = gs.rope_spec(*(spec or (8, 2, 128, 64, 0, 1.0)))
    return gs.lib.rope_rows(ctypes.byref(s), a["B"], a["cap"], a["cu"], a["lens"], a["turns"], a["q"], a["qs"],
                            a["qo"], a["qos"], a["k"], a["ks"], a["ko"], a["kos"], None, None)


def prompts(gs, dims=None, **kw):
    a = dict(B=1, cap=4, cu=64, q=64, qs=1024, k=64, ks=256, v=64, vs=256, o=64, os=1024, rows=4, ws=None, ws_n=0)
    a.update(kw)
    d = gs.attn_dims(*(dims or (8, 2, 128, 0, 0.1)))
    return gs.lib.attn_prompts(ctypes.byref(d), a["B"], a["cap"], a["cu"], a["q"], a["qs"], a["k"], a["ks"], a["v"],
                               a["vs"], a["o"], a["os"], None, a["rows"], a["ws"], a["ws_n"], None, None)


def cache(gs, **kw):
    d = dict(h_q=8, h_kv=2, d=128, page_tokens=64, window=0, num_pages=10, num_layers=2, sm_scale=0.1, kv=4096,
             page_stride=2 * 32768, layer_stride=32768, scale=4096, scale_page_stride=8, scale_layer_stride=4)
    d.update(kw)
    c = gs.kv8_cache()
    for k, v in d.items():
        setattr(c, k, v)
    return c


def chunk(gs, c, **kw):
    a = dict(layer=0, B=1, cap=4, cu=64, lens=64, table=64, pages=4, stride=4, q=64, qs=1024, k=64, ks=256, v=64,
             vs=256, o=64, os=1024, max_len=256, max_rows=4, total=256, ws=64, ws_n=0)
    a.update(kw)
    return gs.lib.kv8_chunk(ctypes.byref(c) if c is not None else None, a["layer"], a["B"], a["cap"], a["cu"],
                            a["lens"], a["table"], a["pages"], a["stride"], a["q"], a["qs"], a["k"], a["ks"], a["v"],
                            a["vs"], a["o"], a["os"], None, a["max_len"], a["max_rows"], a["total"], a["ws"],
                            a["ws_n"], None, None)


def test_rope_arguments(gs):
    for spec in ((8, 2, 0, 64, 0, 1.0), (8, 2, 100, 64, 0, 1.0), (8, 2, 520, 64, 0, 1.0), (8, 2, 128, 0, 0, 1.0),
                 (8, 2, 128, 63, 0, 1.0), (8, 2, 128, 130, 0, 1.0), (-1, 2, 128, 64, 0, 1.0), (0, 0, 128, 64, 0, 1.0),
                 (60000, 6000, 128, 64, 0, 1.0)):
        assert rope(gs, spec) == gs.GDN_ERR_SHAPE, spec
    assert rope(gs, (8, 2, 128, 64, 0, float("nan"))) == gs.GDN_ERR_ARG
    for kw, code in ((dict(B=-1), gs.GDN_ERR_ARG), (dict(B=65536), gs.GDN_ERR_ARG), (dict(cap=-1), gs.GDN_ERR_ARG),
                     (dict(cu=None), gs.GDN_ERR_NULL), (dict(turns=None), gs.GDN_ERR_NULL),
                     (dict(q=None), gs.GDN_ERR_NULL), (dict(qo=None), gs.GDN_ERR_NULL), (dict(k=None), gs.GDN_ERR_NULL),
                     (dict(ko=None), gs.GDN_ERR_NULL), (dict(q=72), gs.GDN_ERR_ARG), (dict(qs=1020), gs.GDN_ERR_ARG),
                     (dict(qs=1016), gs.GDN_ERR_ARG), (dict(kos=248), gs.GDN_ERR_ARG),
                     (dict(qo=64, qos=2048), gs.GDN_ERR_ARG), (dict(ko=64, kos=512), gs.GDN_ERR_ARG)):
        assert rope(gs, **kw) == code, kw
    assert rope(gs, B=0) == gs.GDN_OK and rope(gs, cap=0, q=None, qo=None) == gs.GDN_OK
    assert gs.lib.rope_rows(None, 1, 4, *([64] * 4), 0, 64, 0, 64, 0, 64, 0, None, None) == gs.GDN_ERR_NULL


def test_prompts_arguments(gs):
    for dims in ((8, 2, 96, 0, 0.1), (8, 2, 512, 0, 0.1), (7, 2, 128, 0, 0.1), (8, 0, 128, 0, 0.1), (0, 2, 128, 0, 0.1),
                 (130, 2, 128, 0, 0.1)):
        assert prompts(gs, dims) == gs.GDN_ERR_SHAPE, dims
        assert gs.attn_prompts_workspace_bytes(gs.attn_dims(*dims), 1, 100, 100) == 0
    for dims in ((8, 2, 128, -1, 0.1), (8, 2, 128, 0, float("inf"))):
        assert prompts(gs, dims) == gs.GDN_ERR_ARG, dims
    for kw, code in ((dict(B=-1), gs.GDN_ERR_ARG), (dict(B=65536), gs.GDN_ERR_ARG), (dict(cap=-1), gs.GDN_ERR_ARG),
                     (dict(rows=-1), gs.GDN_ERR_ARG), (dict(rows=(1 << 25) + 1), gs.GDN_ERR_ARG),
                     (dict(cu=None), gs.GDN_ERR_NULL), (dict(q=None), gs.GDN_ERR_NULL), (dict(k=None), gs.GDN_ERR_NULL),
                     (dict(v=None), gs.GDN_ERR_NULL), (dict(o=None), gs.GDN_ERR_NULL), (dict(q=72), gs.GDN_ERR_ARG),
                     (dict(qs=1020), gs.GDN_ERR_ARG), (dict(ks=248), gs.GDN_ERR_ARG), (dict(v=66), gs.GDN_ERR_ARG),
                     (dict(os=1016), gs.GDN_ERR_ARG)):
        assert prompts(gs, **kw) == code, kw
    for kw, code in ((dict(), gs.GDN_ERR_WORKSPACE), (dict(ws=64, ws_n=1000), gs.GDN_ERR_WORKSPACE),
                     (dict(ws=72, ws_n=1 << 40), gs.GDN_ERR_ARG)):
        assert prompts(gs, (4, 1, 128, 0, 0.1), cap=3000, rows=3000, **kw) == code, kw
    for kw in (dict(B=0), dict(cap=0, q=None), dict(rows=0)):
        assert prompts(gs, **kw) == gs.GDN_OK
    for bad in (0, 1_000_000_001):
        d = gs.attn_dims(8, 2, 128, 0, 0.1)
        assert gs.lib.attn_selftest_prompts_timeout(ctypes.byref(d), 1, 4, 64, 64, 1024, 64, 256, 64, 256, 64, 1024, 4,
                                                    None, 0, None, bad, None) == gs.GDN_ERR_ARG


def test_chunk_arguments(gs):
    for kw, code in ((dict(d=96), gs.GDN_ERR_SHAPE), (dict(page_tokens=48), gs.GDN_ERR_SHAPE),
                     (dict(h_q=130, h_kv=2), gs.GDN_ERR_SHAPE), (dict(window=-1), gs.GDN_ERR_ARG),
                     (dict(kv=None), gs.GDN_ERR_NULL), (dict(page_stride=100), gs.GDN_ERR_ARG)):
        assert chunk(gs, cache(gs, **kw)) == code, kw
        assert gs.kv8_chunk_workspace_bytes(cache(gs, **kw), 1, 4, 256, 4, 256) == 0
    assert chunk(gs, None) == gs.GDN_ERR_NULL
    c = cache(gs)
    for kw, code in ((dict(layer=2), gs.GDN_ERR_ARG), (dict(layer=-1), gs.GDN_ERR_ARG), (dict(B=65536), gs.GDN_ERR_ARG),
                     (dict(cap=-1), gs.GDN_ERR_ARG), (dict(pages=-1), gs.GDN_ERR_ARG), (dict(stride=-4), gs.GDN_ERR_ARG),
                     (dict(max_len=-1), gs.GDN_ERR_ARG), (dict(max_rows=-1), gs.GDN_ERR_ARG),
                     (dict(max_len=(1 << 25) - 3), gs.GDN_ERR_ARG), (dict(total=-1), gs.GDN_ERR_ARG),
                     (dict(B=64, max_len=1 << 24, total=1 << 30), gs.GDN_ERR_ARG),
                     (dict(cu=None), gs.GDN_ERR_NULL), (dict(lens=None), gs.GDN_ERR_NULL),
                     (dict(table=None), gs.GDN_ERR_NULL), (dict(q=None), gs.GDN_ERR_NULL),
                     (dict(k=None), gs.GDN_ERR_NULL), (dict(v=None), gs.GDN_ERR_NULL), (dict(o=None), gs.GDN_ERR_NULL),
                     (dict(q=72), gs.GDN_ERR_ARG), (dict(ks=248), gs.GDN_ERR_ARG), (dict(os=1020), gs.GDN_ERR_ARG),
                     (dict(ws=None), gs.GDN_ERR_WORKSPACE), (dict(ws_n=100), gs.GDN_ERR_WORKSPACE),
                     (dict(ws=72, ws_n=1 << 40), gs.GDN_ERR_ARG)):
        assert chunk(gs, c, **kw) == code, kw
    for kw in (dict(B=0), dict(cap=0, q=None), dict(max_rows=0)):
        assert chunk(gs, c, **kw) == gs.GDN_OK


def test_workspace_sizes(gs):
    """A chunk's keys and values in bf16, of no more than the sum of lengths; parts only where SMs would idle."""
    c = cache(gs)
    one = gs.kv8_chunk_workspace_bytes(c, 4, 100, 10000, 50, 12000)
    assert one >= (12000 + 100) * 2 * 128 * 4 and gs.kv8_chunk_workspace_bytes(c, 4, 100, 10000, 50, 1 << 60) > one
    assert gs.kv8_chunk_workspace_bytes(c, 4, 100, 10000, 50, 1 << 60) == \
        gs.kv8_chunk_workspace_bytes(c, 4, 100, 10000, 50, 40000)
    d = gs.attn_dims(32, 8, 128, 0, 0.1)
    assert gs.attn_prompts_workspace_bytes(d, 16, 60000, 4000) == 0
    assert gs.attn_prompts_workspace_bytes(gs.attn_dims(4, 1, 128, 0, 0.1), 1, 3000, 3000) > 0


def test_binding_calls_what_it_names(gs):
    with pytest.raises(gs.GdnError):
        gs.rope_rows(gs.rope_spec(8, 2, 100, 64, 0, 1.0), 1, 4, 64, 64, 64, 64, 1024, 4096, 1024, 64, 256, 4096, 256, 0,
                     stream=0)
    with pytest.raises(gs.GdnError):
        gs.attn_prompts(gs.attn_dims(8, 2, 96, 0, 0.1), 1, 4, 64, 64, 1024, 64, 256, 64, 256, 64, 1024, 0, 4, 0, 0, 0,
                        stream=0)
    with pytest.raises(gs.GdnError):
        gs.kv8_chunk(cache(gs, d=96), 0, 1, 4, 64, 64, 64, 4, 4, 64, 1024, 64, 256, 64, 256, 64, 1024, 0, 256, 4, 256,
                     0, 0, 0, stream=0)


def test_frequencies(gs):
    from speculative_decoding_hybrid_gb300.prefill import rope_frequencies
    f, m = rope_frequencies(64, 10000.0)
    assert m == 1.0 and f[0] == 1.0 and np.allclose(f, [10000.0 ** (-2 * j / 64) for j in range(32)], rtol=1e-15)
    g, m = rope_frequencies(64, 10000.0, "linear", 4.0)
    assert m == 1.0 and np.allclose(g, f / 4, rtol=1e-15)
    g, m = rope_frequencies(64, 10000.0, "base", 8.0)         # the fastest stays, the slowest is divided by the factor
    assert m == 1.0 and g[0] == 1.0 and abs(g[-1] * 8.0 / f[-1] - 1) < 1e-12
    g, m = rope_frequencies(128, 500000.0, "parts", 16.0, trained=8192)
    f, _ = rope_frequencies(128, 500000.0)
    turns = 8192 * f / (2 * math.pi)
    assert abs(m - (1 + 0.1 * math.log(16))) < 1e-15
    assert np.array_equal(g[turns >= 32], f[turns >= 32]) and np.allclose(g[turns <= 1], f[turns <= 1] / 16, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (g[mid] < f[mid]).all() and (g[mid] > f[mid] / 16).all()
    for bad in (dict(rot=0), dict(rot=7), dict(base=1.0), dict(base=float("inf")), dict(factor=0.5),
                dict(scaling="other"), dict(scaling="parts", factor=2.0), dict(rot=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            rope_frequencies(**{**dict(rot=64), **bad})


def test_rope_tables(gs):
    """Turns are the frequencies over 2 pi as fractions of 2^64; given frequencies and refusals."""
    from speculative_decoding_hybrid_gb300.prefill import Rope
    r = Rope(64, 32, base=100.0, device="cpu")
    got = r.turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    assert np.allclose(got * 2 * math.pi, r.frequencies, rtol=1e-15)
    r = Rope(64, 4, device="cpu", frequencies=[0.5, 7.0], magnitude=2.0)   # above a turn a position: modulo one
    assert r.magnitude == 2.0 and abs(float(r.turns.numpy().view(np.uint64)[1]) / 2 ** 64 - (7.0 / (2 * math.pi) - 1)) < 1e-15
    for bad in (dict(d=60), dict(d=520), dict(rot=66), dict(rot=3), dict(frequencies=[1.0]),
                dict(frequencies=[float("nan")] * 32)):
        with pytest.raises(ValueError):
            Rope(**{**dict(d=64, device="cpu"), **bad})
