"""Page tables of the paged cache on the host: reserve, fork, free, compact,
against a model that keeps sets, and their refusals (no GPU)."""
import numpy as np
import pytest

import kv_util as ku


@pytest.fixture(scope="module")
def gs():
    from speculative_decoding_hybrid_gb300 import build
    build.build()
    from speculative_decoding_hybrid_gb300 import binding
    return binding


def state(pool):
    return pool.refcount.copy().tolist(), pool.free_list()


def row(cap=8):
    return np.full(cap, -1, np.int32)


def test_reserve_grows_by_need(gs):
    pool, t = gs.Pool(6), row()
    n, pair = gs.kv8_pages_reserve(pool, t, 0, 0, 1, 16)
    assert (n, pair, t[:1].tolist()) == (1, None, [0])
    n, pair = gs.kv8_pages_reserve(pool, t, n, 1, 15, 16)
    assert (n, pair) == (1, None)
    n, pair = gs.kv8_pages_reserve(pool, t, n, 16, 17, 16)
    assert (n, pair, t[:3].tolist()) == (3, None, [0, 1, 2])
    assert gs.kv8_pages_reserve(pool, t, n, 33, 0, 16) == (3, None)
    assert pool.free_list() == [3, 4, 5]


def test_reserve_is_all_or_nothing(gs):
    pool, t = gs.Pool(3), row()
    n, _ = gs.kv8_pages_reserve(pool, t, 0, 0, 20, 16)
    before = state(pool), t.copy()
    for args, code in (((n, 20, 60, 16), gs.GDN_ERR_NO_SLOT), ((n, 20, 1000, 16), gs.GDN_ERR_ARG),
                       ((n, 40, 1, 16), gs.GDN_ERR_ARG), ((n, -1, 1, 16), gs.GDN_ERR_ARG),
                       ((n, 0, -1, 16), gs.GDN_ERR_ARG), ((n, 0, 1, 48), gs.GDN_ERR_ARG)):
        with pytest.raises(gs.GdnError) as e:
            gs.kv8_pages_reserve(pool, t, *args)
        assert e.value.status == code
    assert state(pool) == before[0] and np.array_equal(t, before[1])
    t[1] = 2                                              # names a page nobody holds
    with pytest.raises(gs.GdnError):
        gs.kv8_pages_reserve(pool, t, n, 20, 1, 16)


def test_fork_shares_whole_pages_and_copies_the_last(gs):
    pool, a, b, c = gs.Pool(10), row(), row(), row()
    n, _ = gs.kv8_pages_reserve(pool, a, 0, 0, 40, 16)
    m, pair = gs.kv8_pages_fork(pool, a, n, 40, 16, b)
    assert m == 3 and b[:2].tolist() == a[:2].tolist() and pair == (int(a[2]), int(b[2])) and b[2] != a[2]
    assert pool.refcount[a[0]] == 2 and pool.refcount[a[2]] == 1
    k, pair = gs.kv8_pages_fork(pool, a, n, 32, 16, c)     # ends with a page: nothing to copy
    assert k == 2 and pair is None and pool.refcount[a[1]] == 3
    # a child that rolls back into a shared page and writes gets its own copy of it
    k, pair = gs.kv8_pages_reserve(pool, c, k, 20, 2, 16)
    assert pair == (int(a[1]), int(c[1])) and pool.refcount[a[1]] == 2 and pool.refcount[c[1]] == 1
    # one that rolls back to a page's first token needs a page, and nothing of the old one
    k, pair = gs.kv8_pages_reserve(pool, b, m, 16, 1, 16)
    assert pair is None and b[1] != a[1] and pool.refcount[a[1]] == 1
    before = state(pool)
    for args in ((a, n, 100, 16, row()), (a, n, -1, 16, row()), (a, n, 40, 16, row(2)), (a, 9, 140, 16, row(9))):
        with pytest.raises(gs.GdnError):
            gs.kv8_pages_fork(pool, *args)
    assert state(pool) == before


def test_free_needs_every_reference(gs):
    pool, t = gs.Pool(4), row()
    n, _ = gs.kv8_pages_reserve(pool, t, 0, 0, 40, 16)
    twice = np.array([t[0], t[0], t[1]], np.int32)
    before = state(pool)
    with pytest.raises(gs.GdnError):
        gs.kv8_pages_free(pool, twice, 3)
    assert state(pool) == before
    gs.kv8_pages_free(pool, t, n)
    assert t.tolist() == [-1] * 8 and sorted(pool.free_list()) == [0, 1, 2, 3]
    with pytest.raises(gs.GdnError):
        gs.kv8_pages_free(pool, np.array([0], np.int32), 1)


def test_compact_refuses_pages_held_elsewhere(gs):
    pool = gs.Pool(8)
    pool.alloc()                                          # held, named by no table
    tables, n = np.full((1, 4), -1, np.int32), np.zeros(1, np.int32)
    n[0], _ = gs.kv8_pages_reserve(pool, tables[0], 0, 0, 40, 16)
    before = state(pool), tables.copy()
    with pytest.raises(gs.GdnError):
        gs.kv8_pages_compact(pool, tables, n)
    assert state(pool) == before[0] and np.array_equal(tables, before[1])


@pytest.mark.parametrize("seed", range(8))
def test_random_life_against_a_model(gs, seed):
    """Contents per page, followed through reserve, append, fork, rollback, free and compact: no request ever
    reads another's token, the pool's counts are the tables', and compaction packs."""
    g = np.random.RandomState(seed)
    T, R, cap, pages = 16, 6, 8, 30
    pool = gs.Pool(pages, free_order=g.permutation(pages))
    tables, n = np.full((R, cap), -1, np.int32), np.zeros(R, np.int32)
    length = [0] * R
    mem = np.full((pages, T), -1, np.int64)               # what the device would hold
    want = [[] for _ in range(R)]
    stamp = 0

    def copy(pair):
        if pair:
            mem[pair[1]] = mem[pair[0]]

    for _ in range(400):
        r, what = g.randint(R), g.randint(10)
        if what < 5:
            new = g.randint(0, 30)
            if length[r] + new > cap * T:
                continue
            try:
                n[r], pair = gs.kv8_pages_reserve(pool, tables[r], int(n[r]), length[r], new, T)
            except gs.GdnError as e:
                assert e.status == gs.GDN_ERR_NO_SLOT
                continue
            copy(pair)
            for _ in range(new):
                assert pool.refcount[tables[r, length[r] // T]] == 1
                mem[tables[r, length[r] // T], length[r] % T] = stamp
                want[r].append(stamp)
                length[r] += 1
                stamp += 1
        elif what < 7:
            s = g.randint(R)
            if n[r] or s == r:
                continue
            m = g.randint(0, length[s] + 1)
            try:
                n[r], pair = gs.kv8_pages_fork(pool, tables[s], int(n[s]), m, T, tables[r])
            except gs.GdnError as e:
                assert e.status == gs.GDN_ERR_NO_SLOT
                continue
            copy(pair)
            length[r], want[r] = m, want[s][:m]
        elif what == 7:
            length[r] = g.randint(0, length[r] + 1)
            want[r] = want[r][:length[r]]
        elif what == 8:
            gs.kv8_pages_free(pool, tables[r], int(n[r]))
            n[r], length[r], want[r] = 0, 0, []
        else:
            src, dst = gs.kv8_pages_compact(pool, tables, n)
            live = len(set(tables[tables >= 0].tolist()))
            assert len(set(dst)) == len(dst) and not set(src) & set(dst) and (src >= live).all() and (dst < live).all()
            assert tables.max(initial=-1) < live and pool.free_list() == list(range(live, pages))
            mem[dst] = mem[src]
            mem[src] = -2
        counts = np.zeros(pages, np.int64)
        for q in range(R):
            np.add.at(counts, tables[q, :n[q]], 1)
            got = [mem[tables[q, t // T], t % T] for t in range(length[q])]
            assert got == want[q]
        assert np.array_equal(counts, pool.refcount)
        assert sorted(pool.free_list()) == np.flatnonzero(counts == 0).tolist()


def test_oracle_rounds_like_its_definition():
    """encode() against a search over all values, scale_for() at its edges."""
    g = np.random.RandomState(0)
    x = np.concatenate([g.standard_normal(500) * 100, g.standard_normal(500) * 0.01, ku.VALUES[:127],
                        (ku.VALUES[:126] + ku.VALUES[1:127]) / 2, [1e9, -1e9]])
    pos = ku.VALUES[:127]
    for v, c in zip(x, ku.encode(x)):
        err = np.abs(np.minimum(abs(v), 448) - pos)
        best = np.flatnonzero(err == err.min())
        assert (c & 127) in best and (len(best) == 1 or (c & 127) % 2 == 0)
        assert c >> 7 == (v < 0)
    assert ku.scale_for(448.0) == 1 and ku.scale_for(448.1) == 2 and ku.scale_for(224.0) == 0.5
    assert ku.scale_for(0.0) == 2.0 ** -100 and ku.scale_for(1e-45) == 2.0 ** -100
