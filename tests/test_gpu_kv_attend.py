"""Attention over the paged 8-bit cache against the fp64 form: head layouts,
page sizes, ragged rows and lengths, windows, empty rows, pieces of any size,
what lies past a request's end, strides, streams and refusals."""
import ctypes

import numpy as np
import pytest
import torch

import kv_util as ku
from gpu_util import build_lib, noted

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def make(cache, rows, seed, k_scale=1.0, stride_pad=0):
    """Packed rows of a fused projection (q, k, v side by side) and their fp64 values."""
    g = np.random.RandomState(seed + 1000)
    R = sum(rows)
    hq, hk, d = cache.h_q, cache.h_kv, cache.d
    x = g.standard_normal((R, (hq + 2 * hk) * d + stride_pad))
    x[:, hq * d:(hq + hk) * d] *= k_scale
    t, f = ku.bf16(x)
    cut = lambda z, a, h: z[:, a:a + h * d].reshape(R, h, d)
    views = lambda z: (cut(z, 0, hq), cut(z, hq * d, hk), cut(z, (hq + hk) * d, hk))
    return t, views(f)


def run(cache, rows, dev, window=0, split=0, layer=0, seed=0, fresh=True, sm_scale=None, max_len=None, pad=0,
        k_scale=1.0, edit=None, want_lse=True):
    R = sum(rows)
    hq, hk, d = cache.h_q, cache.h_kv, cache.d
    t, (q, k, v) = make(cache, rows, seed, k_scale, pad)
    if edit:
        edit(t, q, k, v)
    t = t.to(dev)
    qt = t[:, :hq * d].unflatten(1, (hq, d))
    kt = t[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    vt = t[:, (hq + hk) * d:(hq + 2 * hk) * d].unflatten(1, (hk, d))
    c = ku.gpu_cache(cache, dev, window, sm_scale)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    args = (torch.from_numpy(cache.table).to(dev), torch.tensor(cache.lens, dtype=torch.int32, device=dev),
            torch.from_numpy(cu).to(dev))
    o, lse = c.attend(layer, *args, qt, kt if fresh else None, vt if fresh else None,
                      max_len=max(cache.lens) if max_len is None else max_len, max_rows=max(rows), split_tokens=split,
                      want_lse=want_lse)
    torch.cuda.synchronize()
    return c, o, lse, (q, k, v), cu, args, (qt, kt, vt)


def check(name, cache, rows, dev, window=0, layer=0, fresh=True, sm_scale=None, **kw):
    c, o, lse, (q, k, v), cu, _, _ = run(cache, rows, dev, window=window, layer=layer, fresh=fresh,
                                         sm_scale=sm_scale, **kw)
    assert int(c.status.item()) == 0
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    sc = ku.default_scale(cache.d) if sm_scale is None else float(np.float32(sm_scale))
    for r, n in enumerate(rows):
        a, b = cu[r], cu[r + 1]
        if n == 0:
            continue
        ro, rl, ra, rw = ku.attend_request(cache.dense(r, layer), q[a:b], k[a:b] if fresh else None,
                                           v[a:b] if fresh else None, window, sc)
        ob, lb = ku.attend_bounds(ro, rl, ra, rw, cache.d)
        dead = np.isneginf(rl)
        assert np.array_equal(dead, np.isneginf(lse[a:b])) and not o[a:b][dead].any()
        assert noted("kv attend %s: o" % name, np.max(np.abs(o[a:b] - ro) / ob, initial=0.0)) <= 1.0, (r, n)
        assert noted("kv attend %s: lse" % name,
                     np.max(np.abs(lse[a:b][~dead] - rl[~dead]) / lb[~dead], initial=0.0)) <= 1.0, (r, n)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (6, 2), (16, 2), (8, 8), (24, 1)])
def test_head_layouts(cuda_dev, d, h_q, h_kv):
    cache = ku.Cache([0, 1, 63, 200, 517], h_q, h_kv, d, 64, seed=d + h_q)
    check("heads d=%d" % d, cache, [4, 1, 3, 2, 4], cuda_dev, seed=h_q)


@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_page_sizes_and_lengths(cuda_dev, T, d):
    lens = [1, T - 1, T, T + 1, 127, 128, 129, 255, 256, 257, 3 * T + 5, 900]
    cache = ku.Cache(lens, 4, 2, d, T, seed=T)
    check("pages T=%d d=%d" % (T, d), cache, [1 + i % 4 for i in range(len(lens))], cuda_dev, seed=T)


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 8, 11, 16])
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 1, 128), (16, 2, 256), (5, 5, 64)])
def test_rows(cuda_dev, rows, h_q, h_kv, d):
    cache = ku.Cache([300, 17, 0], h_q, h_kv, d, 32, seed=rows)
    check("rows d=%d" % d, cache, [rows, max(1, rows - 1), rows], cuda_dev, seed=rows)


def test_widest_group(cuda_dev):
    cache = ku.Cache([200], 64, 1, 128, 64, seed=5)
    check("64 query heads a kv head, 16 rows", cache, [16], cuda_dev)


@pytest.mark.parametrize("split", [0, 1, 128, 256, 640, 1 << 20])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_pieces(cuda_dev, split, d):
    cache = ku.Cache([0, 1, 128, 129, 1000, 2500], 6, 2, d, 16, seed=split % 97)
    check("pieces d=%d" % d, cache, [1, 4, 3, 4, 2, 4], cuda_dev, split=split)


@pytest.mark.parametrize("window", [1, 2, 5, 64, 100, 128, 1000])
@pytest.mark.parametrize("fresh", [True, False])
@pytest.mark.parametrize("split", [0, 128])
def test_windows(cuda_dev, window, fresh, split):
    cache = ku.Cache([0, 1, 3, 64, 200, 777], 4, 2, 128, 32, seed=window)
    check("window", cache, [4, 4, 16, 3, 5, 2], cuda_dev, window=window, fresh=fresh, split=split)


def test_cache_only_and_empty_rows(cuda_dev):
    """Without rows of its own a request of length 0 sees nothing: o = 0, lse = -inf."""
    cache = ku.Cache([0, 5, 0, 400], 8, 2, 128, 64, seed=3)
    check("cache only", cache, [2, 3, 1, 4], cuda_dev, fresh=False)
    check("cache only, pieces", cache, [2, 3, 1, 4], cuda_dev, fresh=False, split=128)


def test_requests_without_rows(cuda_dev):
    cache = ku.Cache([70, 5, 300, 9], 8, 2, 128, 64, seed=4)
    check("no rows", cache, [0, 3, 0, 1], cuda_dev)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("split", [0, 128])
def test_bytes_past_the_end_reach_nothing(cuda_dev, d, split):
    """NaN codes past a request's end and pages of others with infinite scales."""
    lens = [0, 1, 31, 33, 130, 255, 700]
    cache = ku.Cache(lens, 4, 2, d, 32, seed=8, fill="garbage")
    check("garbage d=%d" % d, cache, [4, 1, 2, 3, 16, 4, 1], cuda_dev, split=split)
    check("garbage d=%d" % d, cache, [4, 1, 2, 3, 16, 4, 1], cuda_dev, split=split, window=40)


def test_nan_before_the_window_reaches_nothing(cuda_dev):
    cache = ku.Cache([400, 300], 4, 2, 128, 32, seed=9)
    for r, first in ((0, 400 - 99), (1, 300 - 99)):   # row 0 sees positions > len - 100
        for t in range(first):
            cache.kv[cache.table[r, t // 32], :, :, :, t % 32] = 127
    check("nan before the window", cache, [1, 1], cuda_dev, window=100)
    check("nan before the window", cache, [1, 1], cuda_dev, window=100, split=128)


def test_scales_far_apart(cuda_dev):
    """Pages whose keys or values are 2^12 larger or smaller than their neighbours', and a page of zeros."""
    cache = ku.Cache([600], 4, 2, 128, 32, seed=10)
    g = np.random.RandomState(1)
    for j, p in enumerate(cache.table[0]):
        cache.scale[p, :, :, 1] *= 2.0 ** float(g.randint(-12, 13))
        cache.scale[p, :, :, 0] *= 2.0 ** float(g.randint(-12, 1))
        if j == 4:
            cache.kv[p, :, 1] = 0
            cache.scale[p, :, :, 1] = 0
    check("scales far apart", cache, [4], cuda_dev)
    check("scales far apart", cache, [4], cuda_dev, split=128)


@pytest.mark.parametrize("k_scale,sm_scale", [(1.0, 0.0), (1.0, 1.0), (30.0, 0.25), (1e-3, 1.0), (1.0, -0.3)])
def test_score_ranges(cuda_dev, k_scale, sm_scale):
    """Flat scores, scores of +-hundreds (one position takes all, wherever it stands), a negative factor."""
    cache = ku.Cache([700, 40], 8, 2, 128, 64, seed=11)
    cache.scale[:, :, :, 0] *= 2.0 ** float(np.round(np.log2(k_scale)))
    check("score ranges", cache, [4, 4], cuda_dev, sm_scale=sm_scale, k_scale=k_scale)
    check("score ranges", cache, [4, 4], cuda_dev, sm_scale=sm_scale, k_scale=k_scale, split=128)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rising_scores(cuda_dev, d):
    """Every position's score above all before it, by a little and by a lot: the running maximum moves all the time."""
    cache = ku.Cache([900], 2, 1, d, 32, seed=12)
    t = np.arange(900)
    key = np.zeros((900, d))
    key[:, 0] = t * 0.05
    for j, p in enumerate(cache.table[0]):
        part = key[j * 32:(j + 1) * 32]
        s = ku.scale_for(np.abs(part).max())
        cache.kv[p, 0, 0, 0, :len(part)] = ku.encode(part / s)
        cache.scale[p, 0, 0, 0] = s

    def edit(t_, q, k, v):
        t_[:, :] = t_                                   # q = (c, 0, ...): scores rise with the position
        t_[:, :2 * d] = 0
        t_[:, 0], t_[:, d] = 4.0, 0.5
        q[:] = 0
        q[:, 0, 0], q[:, 1, 0] = 4.0, 0.5
    check("rising", cache, [3], cuda_dev, edit=edit, sm_scale=1.0)
    check("rising", cache, [3], cuda_dev, edit=edit, sm_scale=1.0, split=256)


def test_equal_positions_share(cuda_dev):
    """4,000 equal keys under one that scores 9 higher: small weights all alike must not be lost."""
    L = 4000
    cache = ku.Cache([L], 1, 1, 128, 64, seed=13)
    cache.kv[:, :, 0] = 0
    cache.scale[:, :, :, 0] = 1.0
    cache.kv[cache.table[0, 0], 0, 0, 0, 0, 0] = ku.encode(9.0)
    cache.kv[:, :, 1] = ku.encode(1.0)
    cache.kv[cache.table[0, 0], 0, 1, 0, 0] = ku.encode(-1.0)
    cache.scale[:, :, :, 1] = 1.0

    def edit(t, q, k, v):
        t[:, :256] = 0
        t[:, 0] = 1.0
        q[:], k[:] = 0, 0
        q[:, 0, 0] = 1.0
    check("equal positions", cache, [1], cuda_dev, edit=edit, sm_scale=1.0)


def test_rows_do_not_poison_each_other(cuda_dev):
    """A query of NaN, one of infinities and one with a wide range of magnitudes change only their own outputs."""
    cache = ku.Cache([333], 4, 2, 128, 32, seed=14)
    rows = [4]

    def edit(t, q, k, v):
        t[1, :128] = float("nan")
        t[2, 128:256] = float("inf")
        t[3, 0:128:3] *= 2.0 ** -20
    _, o, lse, (q, k, v), cu, _, _ = run(cache, rows, cuda_dev, edit=edit)
    q = q.copy()
    q[3, 0, ::3] *= 2.0 ** -20
    ro, rl, ra, rw = ku.attend_request(cache.dense(0, 0), q, k, v, 0, ku.default_scale(128))
    ob, lb = ku.attend_bounds(ro, rl, ra, rw, 128)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(o[1, 0]).all() and np.isnan(lse[1, 0]) and np.isnan(o[2, 1]).all()
    ok = np.ones((4, 4), bool)
    ok[1, 0] = ok[2, 1] = False
    assert np.max(np.abs(o - ro)[ok] / ob[ok]) <= 1 and np.max(np.abs(lse - rl)[ok] / lb[ok]) <= 1


def test_strides_layers_and_no_lse(cuda_dev):
    """Padded rows, the second of three layers, an output buffer inside a larger one, no log-sum-exp."""
    cache = ku.Cache([150, 20], 4, 2, 128, 32, layers=3, seed=15)
    check("strides", cache, [2, 4], cuda_dev, layer=1, pad=24)
    c, o, lse, _, cu, args, (qt, kt, vt) = run(cache, [2, 4], cuda_dev, layer=2, pad=40)
    big = torch.full((8, 6, 128), 7.0, dtype=torch.bfloat16, device=cuda_dev)
    got, none = c.attend(2, *args, qt, kt, vt, max_len=150, max_rows=4, out=big[1:7, :4])
    assert none is None and torch.equal(got, o)
    big[1:7, :4] = 7.0
    assert (big == 7.0).all()


def test_pinned_pieces_make_bits_independent_of_the_batch(cuda_dev):
    lens, rows = [900, 3000, 10, 1], [4, 2, 3, 1]
    cache = ku.Cache(lens, 8, 2, 128, 64, seed=16)
    c, o, lse, _, cu, (table, length, cu_t), (qt, kt, vt) = run(cache, rows, cuda_dev, split=512)
    for r, n in enumerate(rows):
        a, b = int(cu[r]), int(cu[r + 1])
        one = torch.tensor([0, n], dtype=torch.int32, device=cuda_dev)
        o1, l1 = c.attend(0, table[r:r + 1], length[r:r + 1].clone(), one, qt[a:b], kt[a:b], vt[a:b], max_len=lens[r],
                          max_rows=n, split_tokens=512, want_lse=True)
        assert torch.equal(o1, o[a:b]) and torch.equal(l1, lse[a:b])
    again, _ = c.attend(0, table, length, cu_t, qt, kt, vt, max_len=4000, max_rows=16, split_tokens=512)
    assert torch.equal(again, o)


@pytest.mark.parametrize("d,h_kv,group,rows", [(64, 2, 8, 2), (128, 1, 8, 2), (256, 1, 8, 2), (256, 2, 8, 1),
                                               (64, 1, 4, 4), (128, 2, 16, 4)])
@pytest.mark.parametrize("window", [0, 222])  # 222: row 0 alone sees one position of a tile
def test_pinned_pieces_make_bits_independent_of_max_rows(cuda_dev, d, h_kv, group, rows, window):
    """Scores that grow along the cache move a column's reference again and again, at other tiles than its
    neighbours': how many columns a block has (it goes by max_rows) must not show."""
    lens = [1500, 700]
    cache = ku.Cache(lens, h_kv * group, h_kv, d, 64, seed=23)
    c, o, lse, _, cu, (table, length, cu_t), (qt, kt, vt) = run(cache, [rows, rows], cuda_dev, window=window,
                                                             split=1024)
    for r, n in enumerate(lens):  # keys eight times larger every four pages
        for j in range(-(-n // 64)):
            c.scale[table[r, j].long(), :, :, 0] = 2.0 ** (3 * (j // 4) - 9)
    want = None
    for most in (rows, 4, 8, 16):
        o, lse = c.attend(0, table, length, cu_t, qt, kt, vt, max_len=1500, max_rows=max(rows, most),
                          split_tokens=1024, want_lse=True)
        assert torch.isfinite(lse).all()
        if want is None:
            want = o, lse
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), most
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("d,group,rows,window,page", [
    (64, 2, 8, 0, 16), (64, 4, 8, 70, 32), (64, 4, 16, 0, 64), (128, 4, 4, 40, 64), (128, 8, 4, 0, 16),
    (128, 4, 16, 130, 128), (128, 6, 16, 0, 64), (256, 4, 4, 0, 64), (256, 8, 4, 33, 32), (256, 3, 16, 0, 128)])
def test_many_requests_have_wide_blocks(cuda_dev, d, group, rows, window, page):
    """More requests than CTAs: a block has as many of a request's 16 to 96 columns as it can."""
    g = np.random.RandomState(d + group + rows)
    lens = [int(x) for x in g.randint(0, 300, 160)]
    n = [int(x) for x in g.randint(0, rows + 1, 160)]
    n[7], n[80], lens[80], lens[81] = rows, rows, 0, 256
    check("wide blocks", ku.Cache(lens, group, 1, d, page, seed=31), n, cuda_dev, window=window)


@pytest.mark.parametrize("d,group,rows,lens", [(64, 8, 2, [20000, 100]), (128, 8, 4, [12001, 9000, 30]),
                                               (128, 4, 16, [12000, 127, 9000, 0]), (256, 8, 4, [20010, 3])])
@pytest.mark.parametrize("split", [0, 5000])
def test_long_requests_have_wide_blocks(cuda_dev, d, group, rows, lens, split):
    n = [rows] + [max(1, rows - 1 - i) for i in range(len(lens) - 1)]
    check("wide blocks, long", ku.Cache(lens, 2 * group, 2, d, 64, seed=32), n, cuda_dev, split=split)


def test_another_stream_and_repeats(cuda_dev):
    cache = ku.Cache([2000, 50], 8, 2, 128, 64, seed=17)
    c, o, lse, _, _, args, (qt, kt, vt) = run(cache, [4, 4], cuda_dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [c.attend(0, *args, qt, kt, vt, max_len=2000, max_rows=4, want_lse=True, stream=side) for _ in range(20)]
    side.synchronize()
    for o1, l1 in outs:
        assert torch.equal(o1, o) and torch.equal(l1, lse)


def test_in_a_graph_with_moving_lengths(cuda_dev):
    """Lengths, tables and rows are read on the device: a captured call serves later transactions."""
    cache = ku.Cache([900, 1500], 8, 2, 128, 64, seed=18)
    c, o, _, _, _, (table, length, cu), (qt, kt, vt) = run(cache, [4, 2], cuda_dev, max_len=2000)
    out = torch.empty_like(o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.attend(0, table, length, cu, qt, kt, vt, max_len=2000, max_rows=4, out=out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(0, table, length, cu, qt, kt, vt, max_len=2000, max_rows=4, out=out)
    for lens in ([900, 1500], [3, 1499], [640, 0]):
        length.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        want, _ = c.attend(0, table, length, cu, qt, kt, vt, max_len=2000, max_rows=4)
        assert torch.equal(out, want)
    assert torch.equal(length.cpu(), torch.tensor([640, 0], dtype=torch.int32))


def test_device_refusals_skip_one_request(cuda_dev):
    """A page out of range, a length past max_len, too many rows: that request's outputs stay as they were."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([300, 300, 300, 40], 4, 2, 128, 32, seed=19)
    rows = [2, 2, 2, 2]
    c, o, lse, _, cu, (table, length, cu_t), (qt, kt, vt) = run(cache, rows, cuda_dev)

    def again(tb, ln, cur, split, max_rows=2):
        c.status.zero_()
        out = torch.full_like(o, 5.0)
        c.attend(0, tb, ln, cur, qt, kt, vt, max_len=300, max_rows=max_rows, out=out, split_tokens=split)
        return out, int(c.status.item())

    for split in (0, 128):
        base, st = again(table, length, cu_t, split)
        assert st == 0
        for page in (-1, cache.pages):
            tb = table.clone()
            tb[1, 4] = page                             # the second piece of request 1
            out, st = again(tb, length, cu_t, split)
            assert st == gs.DEV_PAGE_OOR
            assert (out[2:4] == 5.0).all() and torch.equal(out[:2], base[:2]) and torch.equal(out[4:], base[4:])
        for bad in (301, -1):
            ln = length.clone()
            ln[2] = bad
            out, st = again(table, ln, cu_t, split)
            assert st == gs.DEV_ROWS_BAD
            assert (out[4:6] == 5.0).all() and torch.equal(out[:4], base[:4]) and torch.equal(out[6:], base[6:])
        cur = torch.tensor([0, 2, 5, 6, 8], dtype=torch.int32, device=cuda_dev)
        out, st = again(table, length, cur, split)      # request 1 has 3 rows, max_rows is 2
        assert st == gs.DEV_ROWS_BAD and (out[2:5] == 5.0).all() and torch.equal(out[:2], base[:2])
        cur = torch.tensor([0, 2, 4, 6, 9], dtype=torch.int32, device=cuda_dev)
        out, st = again(table, length, cur, split, max_rows=3)   # past the last row
        assert st == gs.DEV_ROWS_BAD and (out[6:] == 5.0).all() and torch.equal(out[:6], base[:6])


def test_offsets_past_32_bits(cuda_dev):
    """Pages whose byte offsets pass 2^32 (a pool of 9 GB)."""
    T, h, d = 64, 2, 256
    pages, layers = 9000, 16
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.fail("needs 30 GB of device memory")
    from speculative_decoding_hybrid_gb300.kvcache import Kv8Cache
    small = ku.Cache([500], 16, h, d, T, layers=1, seed=20)
    kv = torch.zeros((pages, layers, 2, h, T, d), dtype=torch.uint8, device=cuda_dev)
    scale = torch.zeros((pages, layers, h, 2), device=cuda_dev)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    far = [8999 - 3 * i for i in range(8)]
    for j, p in enumerate(far):
        kv[p, 15] = torch.from_numpy(small.kv[small.table[0, j], 0]).to(cuda_dev)
        scale[p, 15] = torch.from_numpy(small.scale[small.table[0, j], 0]).to(cuda_dev)
    assert kv.numel() > 1 << 33
    c0, o, _, _, _, (table, length, cu), (qt, kt, vt) = run(small, [4], cuda_dev)
    c = Kv8Cache(kv, scale, 16, status)
    far_t = torch.tensor([far], dtype=torch.int32, device=cuda_dev)
    got, _ = c.attend(15, far_t, length, cu, qt, kt, vt, max_len=500, max_rows=4)
    assert int(status.item()) == 0 and torch.equal(got, o)


def test_host_refusals(cuda_dev):
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([100], 4, 2, 128, 32, seed=21)
    c, o, _, _, _, (table, length, cu), (qt, kt, vt) = run(cache, [2], cuda_dev)

    def call(**kw):
        a = dict(layer=0, q=qt, k_new=kt, v_new=vt, max_len=100, max_rows=2, split_tokens=0, table=table)
        a.update(kw)
        return c.attend(a["layer"], a["table"], length, cu, a["q"], a["k_new"], a["v_new"], max_len=a["max_len"],
                        max_rows=a["max_rows"], split_tokens=a["split_tokens"])

    for kw in (dict(layer=1), dict(layer=-1), dict(max_rows=17), dict(max_len=-1), dict(split_tokens=-1)):
        with pytest.raises(gs.GdnError):
            call(**kw)
    odd = torch.empty((2, 4 * 128 + 8), dtype=torch.bfloat16, device=cuda_dev)
    with pytest.raises(gs.GdnError):                    # not 16-byte aligned
        call(q=odd[:, 4:516].unflatten(1, (4, 128)))
    for kw in (dict(q=qt.float()), dict(q=qt[:, :2]), dict(k_new=kt[:1]), dict(table=table.long())):
        with pytest.raises(ValueError):
            call(**kw)

    big = ctypes.byref(c.c)
    need = gs.lib.kv8_attend_workspace_bytes(big, 1, 100000, 2, 128)
    assert need > 0
    st = gs.lib.kv8_attend(big, 0, 1, 2, cu.data_ptr(), length.data_ptr(), table.data_ptr(), 4, 4, qt.data_ptr(),
                           qt.stride(0), kt.data_ptr(), kt.stride(0), vt.data_ptr(), vt.stride(0), o.data_ptr(), 512,
                           None, 100000, 2, 128, None, 0, c.status.data_ptr(), None)
    assert st == gs.GDN_ERR_WORKSPACE


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("split", [0, 256])
def test_a_wait_that_runs_out_writes_nothing(cuda_dev, d, split):
    """A copy that never comes: every wait gives up in time, the status says so, outputs stay as they were, and
    the next call is whole again."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([1500, 40, 700], 4, 2, d, 32, seed=22)
    c, o, _, _, _, (table, length, cu), (qt, _, _) = run(cache, [2, 1, 3], cuda_dev, split=split, fresh=False)
    need = gs.kv8_attend_workspace_bytes(c.c, 3, 1500, 3, split)
    ws = torch.empty((max(need, 16),), dtype=torch.uint8, device=cuda_dev)
    out = torch.full_like(o, 5.0)
    gs.kv8_selftest_attend_timeout(c.c, 0, 3, 6, cu, length, table, table.shape[1], table.stride(0), qt, qt.stride(0),
                                   out, out.stride(0), 1500, 3, split, ws, need, c.status, 2_000_000)
    assert int(c.status.item()) == gs.DEV_TIMEOUT and (out == 5.0).all()
    c.status.zero_()
    again, _ = c.attend(0, table, length, cu, qt, None, None, max_len=1500, max_rows=3, split_tokens=split)
    assert int(c.status.item()) == 0 and torch.equal(again, o)


def test_requests_may_share_a_table_row(cuda_dev):
    """One prefix read by several requests through a table of stride 0."""
    cache = ku.Cache([500], 8, 2, 128, 64, seed=23)
    c, _, _, _, _, (table, length, _), _ = run(cache, [4], cuda_dev)
    g = torch.Generator(device=cuda_dev).manual_seed(3)
    q = torch.randn((12, 8, 128), generator=g, device=cuda_dev).to(torch.bfloat16)
    cu = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device=cuda_dev)
    lens = torch.tensor([500, 128, 300], dtype=torch.int32, device=cuda_dev)
    a, _ = c.attend(0, table.expand(3, -1), lens, cu, q, None, None, max_len=500, max_rows=4, split_tokens=256)
    b, _ = c.attend(0, table.repeat(3, 1), lens, cu, q, None, None, max_len=500, max_rows=4, split_tokens=256)
    assert torch.equal(a, b) and int(c.status.item()) == 0


def test_values_that_are_not_finite_reach_only_who_sees_them(cuda_dev):
    """A NaN and an infinity among the new rows' values and a NaN code in the cache inside some rows' window."""
    cache = ku.Cache([300], 4, 2, 128, 32, seed=24)
    t0 = 300 - 99 + 1                                   # window 100: row 0 sees 201.., row 1 from 202, row 2 from 203
    cache.kv[cache.table[0, t0 // 32], 0, 1, 1, t0 % 32, 17] = 127

    def edit(t, q, k, v):
        t[2, (4 + 2) * 128 + 5] = float("nan")          # row 2, kv head 0, element 5
        t[3, (4 + 2) * 128 + 128 + 9] = float("inf")    # row 3, kv head 1, element 9
    for split in (0, 128):
        _, o, lse, (q, k, v), _, _, _ = run(cache, [4], cuda_dev, window=100, edit=edit, split=split)
        x = cache.dense(0, 0)
        x[1, 1, t0, 17] = 0.0
        ro, rl, ra, rw = ku.attend_request(x, q, k, v, 100, ku.default_scale(128))
        ob, lb = ku.attend_bounds(ro, rl, ra, rw, 128)
        got = o.double().cpu().numpy()
        odd = np.zeros(got.shape, bool)
        odd[0:2, 2:4, 17] = True                        # rows 0 and 1 see position t0 = 202
        odd[2:4, 0:2, 5] = True
        assert np.isnan(got[odd]).all()
        assert (got[3, 2:4, 9] == np.inf).all()
        odd[3, 2:4, 9] = True
        assert np.max(np.abs(got - ro)[~odd] / ob[~odd]) <= 1.0
        assert np.max(np.abs(lse.double().cpu().numpy() - rl) / lb) <= 1.0
