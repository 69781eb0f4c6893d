"""Attention of many new rows over the paged 8-bit cache against the fp64 form: head layouts, pages, ragged rows and
lengths, windows, work cut into parts, what lies past a request's end, refusals, streams and graphs."""
import os
import sys

import numpy as np
import pytest
import torch

import kv_util as ku
import prompt_util as pu
from gpu_util import build_lib, noted

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))


def run(cache, rows, dev, window=0, layer=0, seed=0, sm_scale=None, pad=0, edit=None, total=True, table=None,
        max_len=None, max_rows=None, lens=None, out=None, k_scale=1.0):
    hq, hk, d = cache.h_q, cache.h_kv, cache.d
    t, f = pu.rows_of(sum(rows), hq, hk, d, seed, k_scale, pad)
    if edit:
        edit(*pu.split(t, hq, hk, d))
        f = pu.split(t.double().numpy(), hq, hk, d)
    q, k, v = pu.split(t.to(dev), hq, hk, d)
    c = ku.gpu_cache(cache, dev, window, sm_scale)
    cu = pu.cu_of(rows)
    lens = cache.lens if lens is None else lens
    o, lse = c.attend_chunk(layer, torch.from_numpy(cache.table if table is None else table).to(dev),
                            pu.dev32(lens, dev), pu.dev32(cu, dev), q, k, v,
                            max_len=max(cache.lens) if max_len is None else max_len,
                            max_rows=max(rows) if max_rows is None else max_rows,
                            total_len=sum(cache.lens) if total else None, want_lse=True, out=out)
    torch.cuda.synchronize()
    return c, o, lse, f, cu


def compare(name, cache, o, lse, f, cu, layer, window, sc, requests=None):
    q, k, v = f
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for r, (a, b) in enumerate(zip(cu, cu[1:])):
        if a == b or (requests is not None and r not in requests):
            continue
        ro, rl, ra, rw = pu.attend(q[a:b], k[a:b], v[a:b], window, sc, cache.dense(r, layer))
        ob, lb = pu.bounds(ro, rl, ra, rw, cache.d)
        assert noted("chunk %s: o" % name, np.max(np.abs(o[a:b] - ro) / ob)) <= 1.0, (r, b - a)
        assert noted("chunk %s: lse" % name, np.max(np.abs(lse[a:b] - rl) / lb)) <= 1.0, (r, b - a)


def check(name, cache, rows, dev, window=0, layer=0, sm_scale=None, **kw):
    c, o, lse, f, cu = run(cache, rows, dev, window=window, layer=layer, sm_scale=sm_scale, **kw)
    assert int(c.status.item()) == 0
    compare(name, cache, o, lse, f, cu, layer, window,
            ku.default_scale(cache.d) if sm_scale is None else float(np.float32(sm_scale)))
    return o, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (6, 2), (16, 2), (8, 8), (24, 1)])
def test_head_layouts(cuda_dev, d, h_q, h_kv):
    cache = ku.Cache([0, 1, 63, 200, 517], h_q, h_kv, d, 64, seed=d + h_q)
    check("heads d=%d" % d, cache, [40, 1, 0, 130, 17], cuda_dev, seed=h_q)


@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_page_sizes_and_lengths(cuda_dev, T, d):
    lens = [1, T - 1, T, T + 1, 127, 128, 129, 255, 256, 257, 3 * T + 5, 900]
    cache = ku.Cache(lens, 4, 2, d, T, layers=2, seed=T)
    check("pages T=%d d=%d" % (T, d), cache, [1 + 7 * i for i in range(len(lens))], cuda_dev, seed=T, layer=1)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_few_rows_of_long_requests_are_cut(cuda_dev, d):
    cache = ku.Cache([5000, 130, 2500], 4, 1, d, 64, seed=5)
    check("parts d=%d" % d, cache, [20, 17, 33], cuda_dev)
    cache = ku.Cache([9000], 4, 1, d, 64, seed=6)
    check("parts of one d=%d" % d, cache, [3], cuda_dev)


@pytest.mark.parametrize("window", [1, 2, 64, 100, 128, 1000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows(cuda_dev, window, d):
    cache = ku.Cache([0, 1, 3, 64, 200, 777, 2000], 4, 2, d, 32, seed=window)
    check("window d=%d" % d, cache, [40, 4, 170, 30, 5, 20, 300], cuda_dev, window=window)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_wide_scores(cuda_dev, d):
    cache = ku.Cache([700, 100], 4, 2, d, 64, seed=8)
    check("wide d=%d" % d, cache, [150, 40], cuda_dev, sm_scale=2.0)
    check("negative d=%d" % d, cache, [150, 40], cuda_dev, sm_scale=-0.2)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 50])
def test_what_lies_past_the_end(cuda_dev, d, window):
    """NaN codes and infinite scales behind a request's last position and in pages of nobody."""
    lens = [1, 30, 65, 200, 0]
    clean = ku.Cache(lens, 4, 2, d, 32, seed=1)
    dirty = ku.Cache(lens, 4, 2, d, 32, seed=1, fill="garbage")
    rows = [30, 2, 64, 20, 9]
    a = check("clean", clean, rows, cuda_dev, window=window)
    b = check("garbage", dirty, rows, cuda_dev, window=window)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_nan_codes_reach_those_who_see_them(cuda_dev):
    for d in (64, 256):
        cache = ku.Cache([300], 2, 1, d, 64, seed=2)
        clean = run(cache, [100], cuda_dev, window=150, seed=1)[1].cpu()
        page, t = cache.table[0, 210 // 64], 210 % 64
        cache.kv[page, 0, 1, 0, t, 3] = 127                 # a value at position 210: seen from rows 300 .. 359
        o = run(cache, [100], cuda_dev, window=150, seed=1)[1].cpu()
        hit = torch.zeros(o.shape, dtype=torch.bool)
        hit[:60, :, 3] = True
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit])


def test_agrees_with_attend(cuda_dev):
    """16 rows by either call are within both calls' bounds of each other."""
    cache = ku.Cache([700, 20], 8, 2, 128, 64, seed=3)
    c, o, lse, (q, k, v), cu = run(cache, [16, 9], cuda_dev)
    t, _ = pu.rows_of(25, 8, 2, 128, 0)
    qt, kt, vt = pu.split(t.to(cuda_dev), 8, 2, 128)
    o2, l2 = c.attend(0, torch.from_numpy(cache.table).to(cuda_dev), pu.dev32(cache.lens, cuda_dev),
                      pu.dev32(cu, cuda_dev), qt, kt, vt, max_len=700, want_lse=True)
    for r, (a, b) in enumerate(zip(cu, cu[1:])):
        ref = pu.attend(q[a:b], k[a:b], v[a:b], 0, ku.default_scale(128), cache.dense(r, 0))
        both = pu.bounds(*ref, 128)[0] + ku.attend_bounds(*ref, 128)[0]
        assert (np.abs((o - o2)[a:b].double().cpu().numpy()) <= both).all()


def test_bad_requests_are_skipped(cuda_dev):
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([300, 70, 130], 4, 2, 64, 32, seed=4)
    rows = [20, 30, 40]
    cu = pu.cu_of(rows)
    for kw, bits, bad in ((dict(max_len=200), gs.DEV_ROWS_BAD, 0), (dict(max_rows=35), gs.DEV_ROWS_BAD, 2),
                          (dict(lens=[300, -1, 130]), gs.DEV_ROWS_BAD, 1), ("page", gs.DEV_PAGE_OOR, 1),
                          ("negative page", gs.DEV_PAGE_OOR, 0)):
        table = cache.table.copy()
        if kw == "page":
            table[1, 1] = cache.pages
        if kw == "negative page":
            table[0, 0] = -1
        out = torch.full((90, 4, 64), 7.0, dtype=torch.bfloat16, device=cuda_dev)
        c, o, lse, f, _ = run(cache, rows, cuda_dev, table=table, out=out, **(kw if isinstance(kw, dict) else {}))
        assert int(c.status.item()) == bits
        compare("beside bad", cache, o, lse, f, cu, 0, 0, ku.default_scale(64), [r for r in range(3) if r != bad])
        assert (o[cu[bad]:cu[bad + 1]] == 7.0).all()


def test_bad_pages_of_cut_requests(cuda_dev):
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([4000], 2, 1, 128, 64, seed=4)
    for at in (0, 30, 62):
        table = cache.table.copy()
        table[0, at] = 1 << 30
        out = torch.full((17, 2, 128), 7.0, dtype=torch.bfloat16, device=cuda_dev)
        c, o, _, _, _ = run(cache, [17], cuda_dev, table=table, out=out)
        assert int(c.status.item()) == gs.DEV_PAGE_OOR and (o == 7.0).all()


def test_pages_that_no_row_sees_may_be_bad(cuda_dev):
    cache = ku.Cache([500], 2, 1, 64, 32, seed=4)
    o = run(cache, [40], cuda_dev, window=100)[1]
    table = cache.table.copy()
    table[0, :12] = -7                                     # positions below 384; the first row sees 401 and up
    c, o2, _, _, _ = run(cache, [40], cuda_dev, window=100, table=table)
    assert int(c.status.item()) == 0 and torch.equal(o, o2)


def test_more_than_total_len(cuda_dev):
    """A sum of lengths past the host's bound: the requests that fit are served, the others refused."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([100, 90, 10], 2, 1, 64, 32, seed=4)
    rows = [20, 20, 20]
    t, f = pu.rows_of(60, 2, 1, 64, 0)
    q, k, v = pu.split(t.to(cuda_dev), 2, 1, 64)
    c = ku.gpu_cache(cache, cuda_dev)
    out = torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device=cuda_dev)
    o, lse = c.attend_chunk(0, torch.from_numpy(cache.table).to(cuda_dev), pu.dev32(cache.lens, cuda_dev),
                            pu.dev32(pu.cu_of(rows), cuda_dev), q, k, v, max_len=100, max_rows=20, total_len=150,
                            want_lse=True, out=out)
    assert int(c.status.item()) == gs.DEV_ROWS_BAD
    compare("within", cache, o, lse, f, pu.cu_of(rows), 0, 0, ku.default_scale(64), [0])
    assert (o[40:] == 7.0).all()


def test_a_request_that_starts_past_total_len(cuda_dev):
    """The first request fills what the bound leaves to the row: the one behind it is refused, and said to be."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([100, 100], 2, 1, 64, 32, seed=4)
    t, f = pu.rows_of(60, 2, 1, 64, 0)
    q, k, v = pu.split(t.to(cuda_dev), 2, 1, 64)
    c = ku.gpu_cache(cache, cuda_dev)
    out = torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device=cuda_dev)
    o, lse = c.attend_chunk(0, torch.from_numpy(cache.table).to(cuda_dev), pu.dev32(cache.lens, cuda_dev),
                            pu.dev32([0, 40, 60], cuda_dev), q, k, v, max_len=100, max_rows=40, total_len=80,
                            want_lse=True, out=out)
    assert int(c.status.item()) == gs.DEV_ROWS_BAD       # 80 + 60 rows of room: 140 for the first, none for the second
    compare("within", cache, o, lse, f, [0, 40, 60], 0, 0, ku.default_scale(64), [0])
    assert (o[40:] == 7.0).all()


@pytest.mark.parametrize("d,h_q,h_kv", [(64, 1, 1), (64, 2, 1), (128, 2, 1), (256, 4, 1)])
def test_many_requests_of_masked_tiles(cuda_dev, d, h_q, h_kv):
    """More requests than a list's parts and than CTAs, whose units are masked tiles throughout."""
    rows = [256 if i % 3 else 90 + i % 40 for i in range(330)] if d == 64 else [70 + i % 60 for i in range(330)]
    lens = [100 + i % 7 for i in range(330)]
    cache = ku.Cache(lens, h_q, h_kv, d, 128, seed=d)
    check("many d=%d" % d, cache, rows, cuda_dev)


def test_workspace_of_every_request_at_its_longest(cuda_dev):
    cache = ku.Cache([100, 3, 50], 4, 2, 128, 32, seed=4)
    check("no total", cache, [20, 30, 40], cuda_dev, total=False)


def test_an_earlier_calls_workspace_does_not_show(cuda_dev):
    """The same bits whatever the workspace held."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([1000, 3], 4, 1, 64, 32, seed=4)
    t, _ = pu.rows_of(60, 4, 1, 64, 0)
    q, k, v = pu.split(t.to(cuda_dev), 4, 1, 64)
    c = ku.gpu_cache(cache, cuda_dev)
    need = gs.kv8_chunk_workspace_bytes(c.c, 2, 60, 1000, 40, 1003)
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=cuda_dev)
        o = torch.empty((60, 4, 64), dtype=torch.bfloat16, device=cuda_dev)
        table = torch.from_numpy(cache.table).to(cuda_dev)
        gs.kv8_chunk(c.c, 0, 2, 60, pu.dev32([0, 40, 60], cuda_dev), pu.dev32(cache.lens, cuda_dev), table,
                     table.shape[1], table.stride(0), q, q.stride(0), k, k.stride(0), v, v.stride(0), o, 256, None,
                     1000, 40, 1003, ws, need, c.status)
        outs.append(o)
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_streams_and_graphs(cuda_dev):
    cache = ku.Cache([1000, 300], 4, 1, 128, 32, room=[1000, 1300], seed=4)
    t, _ = pu.rows_of(150, 4, 1, 128, 0)
    q, k, v = pu.split(t.to(cuda_dev), 4, 1, 128)
    c = ku.gpu_cache(cache, cuda_dev)
    table, lens, cu = torch.from_numpy(cache.table).to(cuda_dev), pu.dev32(cache.lens, cuda_dev), pu.dev32([0, 50, 150], cuda_dev)
    call = lambda **kw: c.attend_chunk(0, table, lens, cu, q, k, v, max_len=1300, max_rows=150, total_len=2000,
                                       want_lse=True, **kw)
    ref = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(stream=s)
    s.synchronize()
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out, again = call(), call()
    for new in ([1000, 300], [400, 1300], [0, 0]):
        lens.copy_(pu.dev32(new, cuda_dev))
        g.replay()
        ref = call()
        torch.cuda.synchronize()
        for x in (out, again):
            assert torch.equal(x[0], ref[0]) and torch.equal(x[1], ref[1])
    assert int(c.status.item()) == 0


def test_arguments_are_checked(cuda_dev):
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([10], 4, 2, 64, 32, seed=4)
    c = ku.gpu_cache(cache, cuda_dev)
    x = lambda h, n=8, d=64, **kw: torch.zeros((n, h, d), **{**dict(dtype=torch.bfloat16, device=cuda_dev), **kw})
    good = dict(layer=0, table=torch.from_numpy(cache.table).to(cuda_dev), cache_len=pu.dev32([10], cuda_dev),
                cu_rows=pu.dev32([0, 8], cuda_dev), q=x(4), k_new=x(2), v_new=x(2), max_len=10, max_rows=8)
    c.attend_chunk(**good)
    for bad in (dict(q=x(3)), dict(q=x(4, dtype=torch.float16)), dict(k_new=x(2, n=7)), dict(v_new=x(2, d=128)),
                dict(cache_len=good["cache_len"].long()), dict(cu_rows=pu.dev32([0], cuda_dev)),
                dict(table=good["table"].cpu()), dict(out=x(4, n=5))):
        with pytest.raises(ValueError):
            c.attend_chunk(**{**good, **bad})
    for bad in (dict(layer=1), dict(max_len=-1), dict(max_rows=-1), dict(total_len=-1), dict(total_len=1 << 40, max_len=1 << 30)):
        with pytest.raises(gs.GdnError) as e:
            c.attend_chunk(**{**good, **bad})
        assert e.value.status == gs.GDN_ERR_ARG


@pytest.mark.parametrize("d,page_tokens,h_q,h_kv", [(128, 32, 8, 2), (256, 64, 16, 2), (64, 16, 6, 6)])
def test_prompts_in_chunks_then_transactions(cuda_dev, d, page_tokens, h_q, h_kv):
    """Rotation, attention of the first rows and of later chunks, commits and verification together, against the fp64
    forms on a cache that is followed chunk by chunk."""
    import hybrid_decode as hd
    from test_gpu_kv_paged import Follow
    from test_gpu_rope import turned
    h = hd.HybridDecode(2, 1, 2, 900, h_q=h_q, h_kv=h_kv, d=d, page_tokens=page_tokens, seed=d)
    raw = []
    h.rotate = lambda q, k, cu, length, f=h.rotate: (raw.append((q.clone(), k.clone(), int(length[0]))), f(q, k, cu, length))
    f = Follow(h.kv, 2)
    sc = ku.default_scale(d)
    for r, tokens, chunk in ((0, 700, 300), (1, 90, 37)):
        at = 0
        for rows in h.prefill(r, tokens, chunk):
            n = rows[0][0].shape[0]
            for layer, (q, k, v, o) in enumerate(rows):
                q0, k0, first = raw.pop(0)
                assert first == at
                for x0, x in ((q0, q), (k0, k)):
                    x0, got = x0.double().cpu().numpy(), x.double().cpu().numpy()
                    ref = turned(x0, np.arange(at, at + n, dtype=np.float64), h.rope.frequencies, 1.0, d // 2, False)
                    half = d // 4
                    hyp = np.hypot(x0[..., :half], x0[..., half:2 * half])
                    bound = 2.0 ** -8 * np.abs(ref) + 1e-30
                    bound[..., :2 * half] += 2.0 ** -19.9 * np.concatenate([hyp, hyp], -1)
                    assert (np.abs(got - ref) <= bound).all()
                q, k, v = (x.double().cpu().numpy() for x in (q, k, v))
                ref = pu.attend(q, k, v, 0, sc, f.c[r].dense(0, layer) if at else None)
                ob, _ = pu.bounds(*ref, d)
                assert noted("prompts in chunks d=%d" % d, np.max(np.abs(o.double().cpu().numpy() - ref[0]) / ob)) <= 1.0
            f.append(r, [(k, v) for _, k, v, _ in rows])
            at += n
        f.check(h.kv, r)
    seen, accept = h.step([3, 2])
    f.attend("transactions after prompts d=%d: o" % d, 0, seen, 0, 4, [x[3] for x in seen])
    f.attend("transactions after prompts d=%d: o" % d, 1, seen, 4, 7, [x[3] for x in seen])
    assert int(h.vs.status.item()) == 0
