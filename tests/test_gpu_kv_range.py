"""Attention over the paged 8-bit cache where magnitudes lie far apart: queries
and new keys with large channels that the other side is zero in, rows near the
ends of bf16's range, pages with far larger V scales and next to no weight, and
weights whose rounding shows most; against the fp64 form."""
import math

import numpy as np
import pytest
import torch

import kv_util as ku
from gpu_util import build_lib, noted

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def rows_of(cache, n, seed):
    """fp64 q [R, h_q, d], k and v [R, h_kv, d], N(0, 1)."""
    g = np.random.RandomState(seed)
    R = sum(n)
    return tuple(g.standard_normal((R, h, cache.d)) for h in (cache.h_q, cache.h_kv, cache.h_kv))


def check(name, cache, n, q, k, v, dev, window=0, sm_scale=None, split=0, loss=0.0):
    """One call against the fp64 form.  The error budget is kv_util's, with a weight's rounding as the header
    states it: to fp16's 11 bits, 2^-11 of it at most, and to 2^-32 of the largest weight times V scale that the
    row sees (each position's, times its code).  loss: what scores may be off by besides, in powers of two."""
    (qt, q), (kt, k), (vt, v) = ku.bf16(q), ku.bf16(k), ku.bf16(v)
    c = ku.gpu_cache(cache, dev, window, sm_scale)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    o, lse = c.attend(0, torch.from_numpy(cache.table).to(dev), torch.tensor(cache.lens, dtype=torch.int32, device=dev),
                      torch.from_numpy(cu).to(dev), qt.to(dev), kt.to(dev), vt.to(dev), max_len=max(cache.lens),
                      max_rows=max(n), split_tokens=split, want_lse=True)
    assert int(c.status.item()) == 0
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    sc = ku.default_scale(cache.d) if sm_scale is None else float(np.float32(sm_scale))
    worst = [0.0, 0.0]
    for r in range(len(n)):
        a, b = cu[r], cu[r + 1]
        if a == b:
            continue
        ro, rl, ra, rw = ku.attend_request(cache.dense(r, 0), q[a:b], k[a:b], v[a:b], window, sc)
        ob, lb = ku.attend_bounds(ro, rl, ra, rw, cache.d)
        ob = ob + (2.0 ** -12 + 2 * math.log(2) * loss) * ra + floor(cache, r, q[a:b], k[a:b], window, sc)
        lb = lb + math.log(2) * loss
        assert np.isfinite(o[a:b]).all() and np.isfinite(lse[a:b]).all()
        worst[0] = max(worst[0], noted("kv range %s: o" % name, np.max(np.abs(o[a:b] - ro) / ob)))
        worst[1] = max(worst[1], noted("kv range %s: lse" % name, np.max(np.abs(lse[a:b] - rl) / lb)))
    assert worst[0] <= 1.0 and worst[1] <= 1.0, worst


def floor(cache, r, q, k, window, sm_scale):
    """2^-32 max_t(p_t s_t) sum_t |code_t|, over the cached positions a row sees: [n, h_q, d]."""
    L, T, hk = cache.lens[r], cache.T, cache.h_kv
    n, h_q, d = q.shape
    if L == 0:
        return 0.0
    x = cache.dense(r, 0)                                                    # [2, h, L, d]
    ids = cache.table[r, :-(-L // T)]
    sv = np.repeat(cache.scale[ids, 0, :, 1].astype(np.float64).T, T, 1)[:, :L]  # [h, L]
    keys = np.concatenate([x[0], k.transpose(1, 0, 2)], 1)
    z = np.einsum("nhgd,htd->nhgt", q.reshape(n, hk, h_q // hk, d), keys) * sm_scale
    t, at = np.arange(L + n)[None], (L + np.arange(n))[:, None]
    see = (t <= at) & (t > at - window if window else True)
    z = np.where(see[:, None, None, :], z, -np.inf)
    p = np.exp(z - z.max(-1, keepdims=True))
    p = (p / p.sum(-1, keepdims=True))[..., :L]
    codes = np.abs(x[1]) / np.where(sv > 0, sv, 1.0)[..., None]
    top = (p * sv[None, :, None, :]).max(-1)                                 # [n, h, g]
    total = np.einsum("nt,htd->nhd", see[:, :L].astype(float), codes)
    return 2.0 ** -32 * (top[..., None] * total[:, :, None, :]).reshape(n, h_q, d)


LAYOUTS = [(64, 8, 1, 2), (64, 16, 2, 8), (128, 2, 1, 4), (128, 16, 2, 2), (128, 8, 1, 3), (128, 8, 1, 16),
           (256, 8, 1, 1), (256, 16, 2, 4)]


@pytest.mark.parametrize("r", [8, 12, 14, 15, 17, 20, 30, 60, 100])
@pytest.mark.parametrize("d,h_q,h_kv,rows", LAYOUTS)
def test_large_query_channel_under_zero_keys(cuda_dev, d, h_q, h_kv, rows, r):
    """One channel of the queries 2^r times the others; the keys, cached and new, are zero in it."""
    cache = ku.Cache([300, 40, 0], h_q, h_kv, d, 32, seed=r)
    n = [rows, max(1, rows - 1), rows]
    q, k, v = rows_of(cache, n, 100 + r)
    for h in range(h_kv):
        c = (37 * h + 5 * r) % d
        cache.kv[:, :, 0, h, :, c] = 0
        k[:, h, c] = 0
        q[:, h * h_q // h_kv:(h + 1) * h_q // h_kv, c] = 1.5 * 2.0 ** r
    check("large query channel", cache, n, q, k, v, cuda_dev)
    check("large query channel", cache, n, q, k, v, cuda_dev, window=50, split=128)


@pytest.mark.parametrize("r", [13, 16, 24])
@pytest.mark.parametrize("d,h_q,h_kv,rows", LAYOUTS)
def test_many_large_query_channels_under_zero_keys(cuda_dev, d, h_q, h_kv, rows, r):
    """All but an eighth of the channels, anywhere, 2^r times the rest, and only some rows' queries so."""
    cache = ku.Cache([260, 700], h_q, h_kv, d, 64, seed=r)
    n = [rows, rows]
    q, k, v = rows_of(cache, n, 200 + r)
    big = np.random.RandomState(r).permutation(d)[d // 8:]
    cache.kv[..., big] = np.where(np.arange(2)[None, None, :, None, None, None] == 0, 0, cache.kv[..., big])
    k[:, :, big] = 0
    q[::2, ::2][..., big] *= 2.0 ** r
    check("many large query channels", cache, n, q, k, v, cuda_dev)


@pytest.mark.parametrize("r", [8, 12, 14, 17, 20, 60, 100])
@pytest.mark.parametrize("d,h_q,h_kv,rows", LAYOUTS)
def test_large_key_channel_under_zero_queries(cuda_dev, d, h_q, h_kv, rows, r):
    """One channel of some new keys 2^r times the others; the queries are zero in it."""
    cache = ku.Cache([130, 0], h_q, h_kv, d, 32, seed=r)
    n = [rows, rows]
    q, k, v = rows_of(cache, n, 300 + r)
    c = (11 * r) % d
    q[..., c] = 0
    k[::2, :, c] = -1.25 * 2.0 ** r
    check("large key channel", cache, n, q, k, v, cuda_dev, sm_scale=0.25)


@pytest.mark.parametrize("d,h_q,h_kv,rows", [(64, 4, 2, 4), (128, 8, 1, 2), (128, 8, 1, 16), (256, 8, 1, 4)])
def test_large_channels_on_both_sides(cuda_dev, d, h_q, h_kv, rows):
    """Queries large in one channel and new keys in another, each zero in the other's."""
    cache = ku.Cache([70], h_q, h_kv, d, 32, seed=d)
    q, k, v = rows_of(cache, [rows], 400)
    cache.kv[:, :, 0, :, :, 7] = 0
    q[..., 9], k[..., 7] = 0, 0
    q[..., 7] = 2.0 ** 25
    k[..., 9] = 2.0 ** 22
    check("large channels on both sides", cache, [rows], q, k, v, cuda_dev)


@pytest.mark.parametrize("d,h_q,h_kv,rows", [(64, 4, 2, 4), (128, 8, 1, 2), (128, 8, 1, 16), (256, 8, 1, 4)])
def test_ends_of_the_range(cuda_dev, d, h_q, h_kv, rows):
    """Queries and new keys of 1e37 and of 1e-35, the other side as far the other way; zero rows among them."""
    none = ku.Cache([0], h_q, h_kv, d, 32, seed=1)
    q, k, v = rows_of(none, [rows], 500)
    q[0, 0] = 0
    for e in (123, 110, 100, -100, -110, -118):
        check("ends of the range, new keys", none, [rows], q * 2.0 ** e, k * 2.0 ** -(e - 4), v, cuda_dev,
              sm_scale=0.01)
    for e, s in ((122, -94), (100, -80), (-118, 112), (-105, 100)):
        cache = ku.Cache([200], h_q, h_kv, d, 32, seed=2)
        cache.scale[..., 0] = 2.0 ** s                       # keys of about 448 * 2^s at most
        check("ends of the range, cache", cache, [rows], q * 2.0 ** e, k * 2.0 ** (s + 3), v, cuda_dev,
              sm_scale=2.0 ** (-e - s - 9))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_finite_rows_of_the_largest_values_stay_finite(cuda_dev, d):
    """A query of 3e38 in a channel that every key is zero in, over keys of 1e6 elsewhere."""
    cache = ku.Cache([150], 2, 1, d, 32, seed=3)
    cache.kv[:, :, 0, :, :, 3] = 0
    cache.scale[..., 0] = 2.0 ** 13
    q, k, v = rows_of(cache, [2], 600)
    k *= 2.0 ** 13
    k[..., 3] = 0
    q[..., 3] = 3e38
    check("largest values", cache, [2], q, k, v, cuda_dev, sm_scale=2.0 ** -24)


def scaled_page(cache, j, e, score_down, channel=0):
    """Request 0's page j: values 2^e larger, keys that score `score_down` below the others' (queries hold
    1 in `channel`, in which all other keys are zero)."""
    p = cache.table[0, j]
    cache.kv[:, :, 0, :, :, channel] = 0
    cache.kv[p, :, 0] = 0
    cache.kv[p, :, 0, :, :, channel] = ku.encode(-1.0)
    cache.scale[p, :, :, 0] = score_down
    cache.scale[p, :, :, 1] *= 2.0 ** e


@pytest.mark.parametrize("e", [10, 20, 24, 28, 34, 40])
@pytest.mark.parametrize("d,h_q,h_kv,rows", [(64, 8, 1, 1), (128, 8, 1, 2), (128, 16, 2, 8), (256, 8, 1, 4)])
def test_large_values_without_weight(cuda_dev, d, h_q, h_kv, rows, e):
    """A page whose values are 2^e larger takes next to no weight: the others make the output, wherever it lies."""
    for j in (0, 5, 18):
        cache = ku.Cache([600], h_q, h_kv, d, 32, seed=e)
        scaled_page(cache, j, e, 64.0)
        q, k, v = rows_of(cache, [rows], 700 + e)
        q[..., 0], k[..., 0] = 1.0, 0.0
        for split in (0, 128):
            check("large values without weight", cache, [rows], q, k, v, cuda_dev, sm_scale=1.0, split=split)


@pytest.mark.parametrize("e", [16, 32])
def test_large_values_of_any_weight(cuda_dev, e):
    """The same with a weight that makes up for the size, or leaves a part of it."""
    for down in (0.5 * e, 0.6931471805599453 * e, 1.2 * e):
        cache = ku.Cache([600], 8, 1, 128, 32, seed=e)
        scaled_page(cache, 7, e, float(np.float32(down)))
        q, k, v = rows_of(cache, [2], 800 + e)
        q[..., 0], k[..., 0] = 1.0, 0.0
        check("large values of any weight", cache, [2], q, k, v, cuda_dev, sm_scale=1.0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e", [24, 40])
def test_large_values_that_other_rows_see(cuda_dev, d, e):
    """Row 0 alone sees the last position of a page whose values are 2^e larger; the rows after it see none."""
    T, L, window = 32, 400, 113                         # row 0 sees positions from 288 = 9 * 32 on
    cache = ku.Cache([L], 8, 1, d, T, seed=e)
    cache.scale[cache.table[0, 8], :, :, 1] *= 2.0 ** e  # positions 256 .. 287
    q, k, v = rows_of(cache, [4], 900)
    for w in (window, window + 1, window + 2):
        for split in (0, 128):
            check("large values that others see", cache, [4], q, k, v, cuda_dev, window=w, split=split)


def test_values_that_rise_by_pages(cuda_dev):
    """V scales that rise page by page, 2^40 in all, under scores that fall as fast, rise, or stay."""
    for fall in (-1.5, 0.0, 0.6931471805599453, 1.0, 2.0):
        for sign in (1, -1):
            cache = ku.Cache([640], 8, 1, 128, 32, seed=40)
            cache.kv[:, :, 0, :, :, 0] = 0
            for j, p in enumerate(cache.table[0]):
                x = sign * 2.0 * j
                cache.kv[p, :, 0] = 0
                cache.kv[p, :, 0, :, :, 0] = ku.encode(-1.0 if fall * x > 0 else 1.0)
                cache.scale[p, :, :, 0] = max(2.0 ** -20, abs(fall * x))
                cache.scale[p, :, :, 1] *= 2.0 ** x
            q, k, v = rows_of(cache, [3], 41)
            q[..., 0], k[..., 0] = 1.0, 0.0
            check("values that rise by pages", cache, [3], q, k, v, cuda_dev, sm_scale=1.0)
            check("values that rise by pages", cache, [3], q, k, v, cuda_dev, sm_scale=1.0, split=256)


def test_pages_of_zeros_before_the_others(cuda_dev):
    """A first tile of values zero (the smallest scale there is) that scores highest, then ordinary pages."""
    cache = ku.Cache([700], 8, 1, 128, 32, seed=42)
    cache.kv[:, :, 0, :, :, 0] = 0
    for p in cache.table[0, :4]:
        cache.kv[p] = 0
        cache.kv[p, :, 0, :, :, 0] = ku.encode(20.0)
        cache.scale[p, :, :, 0], cache.scale[p, :, :, 1] = 1.0, 2.0 ** -100
    q, k, v = rows_of(cache, [2], 43)
    q[..., 0], k[..., 0] = 1.0, 0.0
    check("pages of zeros first", cache, [2], q, k, v, cuda_dev, sm_scale=1.0)
    check("pages of zeros first", cache, [2], q, k, v, cuda_dev, sm_scale=1.0, split=256)


def test_a_late_position_that_takes_all(cuda_dev):
    """One late position outweighs all others by less than moves a reference, so that its weight is rounded where
    it is no power of two: by up to 2^-11, which the unrounded sum does not share."""
    L = 300
    cache = ku.Cache([L], 8, 1, 128, 32, seed=44)
    cache.kv[:, :, 0] = 0
    cache.scale[..., 0] = 1.0
    cache.kv[cache.table[0, 8], :, 0, :, 10, 0] = ku.encode(1.0)          # position 266, in the third tile
    cache.kv[cache.table[0, 0], :, 0, :, 0, 1] = ku.encode(1.0)           # and position 0, the reference
    q, k, v = rows_of(cache, [16], 45)
    q[:], k[:] = 0, 0
    q[..., 1] = 60.0
    q[..., 0] = 60.0 + 4.9 + 0.62 * np.arange(128).reshape(16, 8) / 128   # bf16 steps of 0.5 round these
    q[..., 2:] = 0
    check("a late position takes all", cache, [16], q, k, v, cuda_dev, sm_scale=1.0)
    q[..., 0] = 4.9 + 0.62 * np.arange(128).reshape(16, 8) / 128
    q[..., 1] = 0
    cache.scale[:] = 1.0
    check("a late position takes all", cache, [16], q, k, v, cuda_dev, sm_scale=1.0)


@pytest.mark.parametrize("seed", range(48))
def test_any_shape_and_range(cuda_dev, seed):
    """Drawn sizes, masks and cuts with drawn channels, all but a few of them or one, 2^5 to 2^60 above the others
    on one side and zero on the other, and V scales 2^40 apart.  Scores may be off by the 2^-14 that the header
    gives each of the two sides, and sum to nearly nothing."""
    g = np.random.RandomState(1000 + seed)
    pick = lambda *x: x[g.randint(len(x))]
    d, h, group, page = pick(64, 128, 256), pick(1, 2, 4), pick(1, 2, 3, 4, 8, 16), pick(16, 32, 64, 128)
    B, most = pick(1, 2, 3, 8, 40), pick(1, 2, 3, 4, 7, 16)
    hi = pick(3, 50, 130, 400, 1500) if B <= 8 else pick(3, 50, 200)
    lens, rows = [int(x) for x in g.randint(0, hi + 1, B)], [int(x) for x in g.randint(0, most + 1, B)]
    rows[0] = most
    cache = ku.Cache(lens, h * group, h, d, page, seed=seed, fill=pick("normal", "garbage"))
    q, k, v = rows_of(cache, rows, seed)
    if seed % 4 != 3:
        big = g.permutation(d)[:pick(1, d // 2, d - 4, d - 1)]
        keys = cache.kv[:, :, 0]
        keys[..., big] = np.where((keys[..., big] & 127) == 127, keys[..., big], 0)
        k[..., big] = 0
        q[..., big] *= np.where(g.rand(*q.shape[:2]) < 0.7, 2.0 ** float(g.randint(5, 60)), 1.0)[..., None]
    if seed % 4 >= 2:
        c = int(g.randint(d))
        q[..., c] = 0
        k[..., c] *= np.where(g.rand(*k.shape[:2]) < 0.5, 2.0 ** float(g.randint(5, 60)), 1.0)
    if seed % 2:
        some = np.isfinite(cache.scale[..., 1])
        cache.scale[..., 1] *= np.where(some, 2.0 ** g.randint(-20, 21, some.shape), 1.0)
    check("any shape and range", cache, rows, q, k, v, cuda_dev, window=pick(0, 0, 5, 60, 129, 300),
          split=pick(0, 0, 128, 512), loss=2.0 ** -13)


@pytest.mark.parametrize("d,h_kv,group", [(64, 2, 8), (128, 1, 8), (256, 2, 4)])
def test_bits_of_such_rows_do_not_go_by_their_neighbours(cuda_dev, d, h_kv, group):
    """With given cuts a request's bits are its own, whether a row beside it, in its block or not, is summed from
    its elements, and however wide the blocks are."""
    h_q, lens, n = h_kv * group, [900, 300, 40], [4, 2, 3]
    cache = ku.Cache(lens, h_q, h_kv, d, 32, seed=d)
    cache.kv[:, :, 0, :, :, 5] = 0
    q, k, v = rows_of(cache, n, d)
    k[..., 5] = 0
    q[1, 1, 5], q[4, 0, 5], q[6, h_q - 1, 5] = 2.0 ** 20, 2.0 ** 30, 2.0 ** 90
    qt, kt, vt = (ku.bf16(x)[0].to(cuda_dev) for x in (q, k, v))
    c = ku.gpu_cache(cache, cuda_dev)
    table = torch.from_numpy(cache.table).to(cuda_dev)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)
    run = lambda r, a, b, most: c.attend(0, table[r], ints(*[lens[i] for i in range(3)][r]),
                                         ints(*np.concatenate([[0], np.cumsum(n[r])]).tolist()), qt[a:b], kt[a:b],
                                         vt[a:b], max_len=900, max_rows=most, split_tokens=256, want_lse=True)
    o, lse = run(slice(0, 3), 0, 9, 4)
    for most in (8, 16):
        o1, l1 = run(slice(0, 3), 0, 9, most)
        assert torch.equal(o1, o) and torch.equal(l1, lse)
    for r, (a, b) in enumerate(((0, 4), (4, 6), (6, 9))):
        o1, l1 = run(slice(r, r + 1), a, b, n[r])
        assert torch.equal(o1, o[a:b]) and torch.equal(l1, lse[a:b])
    # the other rows' bits are those they have without such a row
    q[1, 1, 5] = q[4, 0, 5] = q[6, h_q - 1, 5] = 0
    qt = ku.bf16(q)[0].to(cuda_dev)
    o1, l1 = run(slice(0, 3), 0, 9, 4)
    same = torch.ones((9, h_q), dtype=torch.bool, device=cuda_dev)
    same[1, 1] = same[4, 0] = same[6, h_q - 1] = False
    assert torch.equal(o1[same], o[same]) and torch.equal(l1[same], lse[same])
