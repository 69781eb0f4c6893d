"""The commit of rows into the paged 8-bit cache, bit for bit against its
definition in fp64, and page copies."""
import numpy as np
import pytest
import torch

import kv_util as ku
from gpu_util import build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def append(cache, rows, dev, accept=None, layer=0, seed=0, scale=1.0, edit=None, pad=0, max_rows=None, c=None):
    """Appends to the GPU copy and to `cache` itself; -> the GPU handle."""
    g = np.random.RandomState(seed + 77)
    R, h, d = sum(rows), cache.h_kv, cache.d
    x = g.standard_normal((R, 2 * h * d + pad)) * scale
    if edit:
        edit(x)
    t, f = ku.bf16(x)
    t = t.to(dev)
    c = ku.gpu_cache(cache, dev) if c is None else c
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    acc = None if accept is None else torch.tensor(accept, dtype=torch.int32, device=dev)
    c.append(layer, torch.from_numpy(cache.table).to(dev), torch.tensor(cache.lens, dtype=torch.int32, device=dev),
             torch.from_numpy(cu).to(dev), t[:, :h * d].unflatten(1, (h, d)),
             t[:, h * d:2 * h * d].unflatten(1, (h, d)), accept_len=acc,
             max_rows=max(rows) if max_rows is None else max_rows)
    torch.cuda.synchronize()
    k, v = f[:, :h * d].reshape(R, h, d), f[:, h * d:2 * h * d].reshape(R, h, d)
    for r, n in enumerate(rows):
        n = n if accept is None else accept[r] + 1
        if n > 0:
            ku.append_request(cache, r, layer, k[cu[r]:cu[r] + n], v[cu[r]:cu[r] + n])
    return c


def same(c, cache):
    got = c.kv.cpu().numpy()
    nan = np.isnan(ku.VALUES[got]) & np.isnan(ku.VALUES[cache.kv])
    zero = (ku.VALUES[got] == 0) & (ku.VALUES[cache.kv] == 0)
    assert np.array_equal(np.where(nan | zero, 0, got), np.where(nan | zero, 0, cache.kv))
    assert np.array_equal(c.scale.cpu().numpy(), cache.scale)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T", [16, 32, 64, 128])
def test_rows_into_fresh_and_held_pages(cuda_dev, T, d):
    lens = [0, 1, T - 1, T, T + 1, 3 * T - 2, 5]
    rows = [1, 4, 3, 16, 2, 4, 16]
    cache = ku.Cache(lens, 4, 2, d, T, room=[a + n for a, n in zip(lens, rows)], seed=T + d)
    same(append(cache, rows, cuda_dev), cache)


@pytest.mark.parametrize("scale", [1e-6, 0.05, 1.0, 40.0, 1e5])
def test_growing_and_shrinking_magnitudes(cuda_dev, scale):
    """New rows far smaller or larger than what the page holds: the earlier codes move with the scale."""
    lens = [3, 10, 31, 0, 40]
    cache = ku.Cache(lens, 3, 3, 128, 32, room=[a + 8 for a in lens], seed=int(scale * 10) % 97)
    same(append(cache, [4, 4, 4, 4, 4], cuda_dev, scale=scale), cache)


def test_row_by_row_grows_again_and_again(cuda_dev):
    cache = ku.Cache([0, 7], 2, 2, 64, 32, room=[40, 47], seed=2)
    c = None
    for step in range(20):
        c = append(cache, [1, 2], cuda_dev, seed=step, scale=2.0 ** (step % 7 - 3) * 1.3 ** step, c=c)
        cache.lens = [cache.lens[0] + 1, cache.lens[1] + 2]
        same(c, cache)


def test_every_value_rounds_to_nearest_even(cuda_dev):
    """All bf16 values between two powers of two over e4m3's whole range, ties among them."""
    bits = np.arange(0x3b00, 0x43e1)                       # 2^-9 .. 448 and a bit more
    vals = torch.from_numpy(bits.astype(np.int32)).to(torch.int16).view(torch.bfloat16).double().numpy()
    vals = vals[vals <= 448.0]
    n = -(-len(vals) // 128)
    flat = np.zeros(n * 128)
    flat[:len(vals)] = vals

    def edit(x):
        x[:, :128] = flat.reshape(n, 128)
        x[:, 128:] = -flat.reshape(n, 128)
        x[:, 0] = 448.0
        x[:, 128] = -448.0
    cache = ku.Cache([0], 1, 1, 128, 16, room=[n], seed=3)
    same(append(cache, [n], cuda_dev, edit=edit), cache)


def test_zeros_infinities_and_nan(cuda_dev):
    def edit(x):
        x[0:4] = 0.0                                       # a page of zeros takes the least scale
        x[4, 3], x[5, 70], x[6, 5] = np.inf, -np.inf, np.nan
        x[8:12] = np.nan
        x[12:16] = np.inf
        x[16:20] = 1e-38                                   # subnormal beside the least scale
        x[20:24] = 3e38
    cache = ku.Cache([0] * 6, 2, 1, 64, 16, room=[4] * 6, seed=4)
    same(append(cache, [4] * 6, cuda_dev, edit=edit), cache)


def test_prompts(cuda_dev):
    lens, rows = [0, 37, 64, 0], [1000, 333, 1, 129]
    cache = ku.Cache(lens, 8, 4, 128, 64, room=[a + n for a, n in zip(lens, rows)], seed=5)
    same(append(cache, rows, cuda_dev), cache)
    cache = ku.Cache(lens, 8, 2, 256, 128, room=[a + n for a, n in zip(lens, rows)], seed=6)
    same(append(cache, rows, cuda_dev), cache)


def test_accept_lengths_layers_and_strides(cuda_dev):
    """Only the accepted rows of the second layer; a refused request (-1) and one without rows change nothing."""
    lens, rows = [30, 31, 0, 64, 9], [4, 4, 4, 16, 0]
    cache = ku.Cache(lens, 4, 2, 128, 32, layers=3, room=[a + n for a, n in zip(lens, rows)], seed=7)
    same(append(cache, rows, cuda_dev, accept=[0, 3, -1, 9, -1], layer=1, pad=40), cache)


def test_appending_twice_changes_nothing_more(cuda_dev):
    cache = ku.Cache([20, 5], 2, 2, 128, 32, room=[36, 9], seed=8)
    c = append(cache, [16, 4], cuda_dev)
    kv, sc = cache.kv.copy(), cache.scale.copy()
    c = append(cache, [16, 4], cuda_dev, c=c)
    assert np.array_equal(kv, cache.kv) and np.array_equal(sc, cache.scale)
    same(c, cache)


def test_device_refusals(cuda_dev):
    from speculative_decoding_hybrid_gb300 import binding as gs
    lens, rows = [20, 5, 7], [4, 4, 4]
    cache = ku.Cache(lens, 2, 2, 128, 32, room=[40, 40, 40], seed=9)
    c = ku.gpu_cache(cache, cuda_dev)
    x = torch.randn((12, 2, 128), device=cuda_dev).to(torch.bfloat16)
    table = torch.from_numpy(cache.table).to(cuda_dev)
    length = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    cu = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device=cuda_dev)
    before = c.kv.clone(), c.scale.clone()

    def untouched(r):
        ids = table[r].long()
        ids = ids[(ids >= 0) & (ids < cache.pages)]
        return torch.equal(c.kv[ids], before[0][ids]) and torch.equal(c.scale[ids], before[1][ids])

    acc = torch.tensor([3, 4, 0], dtype=torch.int32, device=cuda_dev)
    c.append(0, table, length, cu, x, x, accept_len=acc, max_rows=4)
    assert int(c.status.item()) == gs.DEV_ACCEPT_BAD and untouched(1) and not untouched(0) and not untouched(2)
    c.kv.copy_(before[0]), c.scale.copy_(before[1]), c.status.zero_()
    bad = table.clone()
    bad[2, 0] = cache.pages
    c.append(0, bad, length, cu, x, x, max_rows=4)
    assert int(c.status.item()) == gs.DEV_PAGE_OOR and untouched(2) and not untouched(1)
    c.kv.copy_(before[0]), c.scale.copy_(before[1]), c.status.zero_()
    for ln in ([20, -1, 7], [20, 1 << 20, 7]):
        c.append(0, table, torch.tensor(ln, dtype=torch.int32, device=cuda_dev), cu, x, x, max_rows=4)
        assert int(c.status.item()) == gs.DEV_ROWS_BAD and untouched(1)
        c.status.zero_()
    c.kv.copy_(before[0]), c.scale.copy_(before[1])
    c.append(0, table, length, cu, x, x, max_rows=3)         # four rows, the caller said three
    assert int(c.status.item()) == gs.DEV_ROWS_BAD and torch.equal(c.kv, before[0])
    c.status.fill_(gs.DEV_TIMEOUT)                           # an earlier wait ran out: nothing is committed
    c.append(0, table, length, cu, x, x, max_rows=4)
    assert torch.equal(c.kv, before[0]) and torch.equal(c.scale, before[1])
    with pytest.raises(gs.GdnError):
        c.append(1, table, length, cu, x, x)
    with pytest.raises(ValueError):
        c.append(0, table, length, cu, x[:, :1], x)


@pytest.mark.parametrize("T,h,d,layers", [(16, 1, 64, 1), (64, 2, 256, 10), (32, 5, 128, 3)])
def test_copy_pages(cuda_dev, T, h, d, layers):
    from speculative_decoding_hybrid_gb300 import binding as gs
    n = 40
    cache = ku.Cache([0], h, h, d, T, layers=layers, spare=n, seed=T)
    c = ku.gpu_cache(cache, cuda_dev)
    kv, sc = c.kv.clone(), c.scale.clone()
    src, dst = [3, 3, 9, 12, 20], [30, 31, 1, 12, 39]
    kv[dst], sc[dst] = kv[src], sc[src]
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)
    c.copy_pages(t(src), t(dst))
    assert torch.equal(c.kv, kv) and torch.equal(c.scale, sc) and int(c.status.item()) == 0
    c.copy_pages(t([-1, 4, n, 5]), t([0, n, 2, 6]))
    kv[6], sc[6] = kv[5], sc[5]
    assert torch.equal(c.kv, kv) and torch.equal(c.scale, sc) and int(c.status.item()) == gs.DEV_PAGE_OOR
    c.copy_pages(t([]), t([]))
    with pytest.raises(ValueError):
        c.copy_pages(t([1]), t([1, 2]))


def test_copy_of_a_layer_inside_a_wider_pool(cuda_dev):
    """Pages with room between them, as when the cache is a part of a larger allocation."""
    from speculative_decoding_hybrid_gb300.kvcache import Kv8Cache
    wide = torch.randint(0, 120, (12, 4, 2, 2, 16, 64), dtype=torch.uint8, device=cuda_dev)
    sc = torch.rand((12, 4, 2, 2), device=cuda_dev)
    kv, s = wide[:, 1:3], sc[:, 1:3]
    want, want_s = wide.clone(), sc.clone()
    want[7, 1:3], want_s[7, 1:3] = wide[2, 1:3], sc[2, 1:3]
    c = Kv8Cache(kv, s, 2, torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    c.copy_pages(*(torch.tensor([x], dtype=torch.int32, device=cuda_dev) for x in (2, 7)))
    assert torch.equal(wide, want) and torch.equal(sc, want_s)


@pytest.mark.parametrize("B", [3, 40])
def test_ragged_prompts_of_many_requests(cuda_dev, B):
    """Rows from none to hundreds, the pages counted over all requests."""
    g = np.random.RandomState(B)
    rows = [int(x) for x in g.choice([0, 1, 2, 17, 60, 333], B)]
    rows[-1] = 700
    lens = [int(x) for x in g.randint(0, 50, B)]
    cache = ku.Cache(lens, 2, 2, 64, 16, room=[a + n for a, n in zip(lens, rows)], seed=10)
    accept = [n - 1 if i % 3 else max(-1, n - 5) for i, n in enumerate(rows)]
    same(append(cache, rows, cuda_dev, accept=accept), cache)


def test_rows_named_twice(cuda_dev):
    """Requests whose rows overlap (the table goes back) take more pages than the rows would: all are written,
    the request that goes back is refused."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    n = 400
    cache = ku.Cache([0, 0, 0, 5], 1, 1, 64, 16, room=[n, 1, n, 5 + n], seed=11)
    g = np.random.RandomState(12)
    t, f = ku.bf16(g.standard_normal((n, 2, 64)))
    t = t.to(cuda_dev)
    c = ku.gpu_cache(cache, cuda_dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)
    k, v = t[:, :1], t[:, 1:]
    cu = i32([0, n, 0, n, n])                                # request 1 has -n rows, 2 request 0's, 3 none
    c.append(0, torch.from_numpy(cache.table).to(cuda_dev), i32(cache.lens), cu, k, v, max_rows=n)
    assert int(c.status.item()) == gs.DEV_ROWS_BAD
    c.status.zero_()
    for r in (0, 2):
        ku.append_request(cache, r, 0, f[:, :1], f[:, 1:])
    same(c, cache)
