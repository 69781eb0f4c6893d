"""Units that are cut into parts: values and keys that are not finite in any part, what the workspace held before, more
than 32 parts, scores of -inf throughout a part, and a wait that runs out before the join."""
import ctypes

import numpy as np
import pytest
import torch

import kv_util as ku
import prompt_util as pu
from gpu_util import build_lib, noted

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def prompt_workspace(h_q, h_kv, d, n, window=0):
    """Its bytes, and how many parts a unit has at most."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    need = gs.attn_prompts_workspace_bytes(gs.attn_dims(h_q, h_kv, d, window, 0.1), 1, n, n)
    stages = 1 if d == 256 else 2
    per = stages * (128 // (h_q // h_kv))
    units = h_kv * min(-(-n // per), n // per + 1)
    return need, round((need / units - 32) / (stages * 128 * (d * 4 + 8)))


def chunk_workspace(c, cache, rows):
    from speculative_decoding_hybrid_gb300 import binding as gs
    L = cache.lens[0]
    need = gs.kv8_chunk_workspace_bytes(c.c, 1, rows, L, rows, L)
    dense = (L + rows) * cache.h_kv * cache.d * 4
    stages = 1 if cache.d == 256 else 2
    per = stages * (128 // (cache.h_q // cache.h_kv))
    units = cache.h_kv * min(-(-rows // per), rows // per + 1)
    return need, round(((need - dense) / units - 32) / (stages * 128 * (cache.d * 4 + 8)))


def prompt(t, h_q, h_kv, d, dev, window=0):
    from speculative_decoding_hybrid_gb300.prefill import attend_prompts
    q, k, v = pu.split(t.to(dev), h_q, h_kv, d)
    n = t.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    o, lse = attend_prompts(q, k, v, pu.dev32([0, n], dev), n, status, window=window, want_lse=True)
    assert int(status.item()) == 0
    return o.cpu(), lse.cpu()


@pytest.mark.parametrize("d,h_q,h_kv", [(64, 4, 1), (128, 4, 1), (256, 2, 1)])
def test_values_that_are_not_finite_in_a_prompt(cuda_dev, d, h_q, h_kv):
    """In the first part, a middle one and the last, masked one: the rows that see them and no other bit."""
    n = 2000
    need, parts = prompt_workspace(h_q, h_kv, d, n)
    assert need > 0 and parts >= 3
    t, _ = pu.rows_of(n, h_q, h_kv, d, 3)
    clean, lse = prompt(t, h_q, h_kv, d, cuda_dev)
    for at in (0, 3, 127, 128, 700, 1101, 1920, 1983, n - 2, n - 1):
        for what in (float("nan"), float("inf"), float("-inf")):
            x = t.clone()
            pu.split(x, h_q, h_kv, d)[2][at, 0, 5] = what
            o, l = prompt(x, h_q, h_kv, d, cuda_dev)
            hit = torch.zeros(o.shape, dtype=torch.bool)
            hit[at:, :, 5] = True
            assert not torch.isfinite(o[hit]).any() and torch.equal(o[~hit], clean[~hit]) and torch.equal(l, lse)
            if what == float("inf"):
                assert not (o[hit] == -what).any()
        x = t.clone()
        pu.split(x, h_q, h_kv, d)[1][at, 0, 5] = float("nan")
        o, l = prompt(x, h_q, h_kv, d, cuda_dev)
        assert torch.isnan(o[at:]).all() and torch.isnan(l[at:]).all()
        assert torch.equal(o[:at], clean[:at]) and torch.equal(l[:at], lse[:at])


def chunk(cache, t, dev, window=0, table=None):
    c = ku.gpu_cache(cache, dev, window)
    q, k, v = pu.split(t.to(dev), cache.h_q, cache.h_kv, cache.d)
    L, n = cache.lens[0], t.shape[0]
    o, lse = c.attend_chunk(0, torch.from_numpy(cache.table).to(dev), pu.dev32([L], dev), pu.dev32([0, n], dev), q, k, v,
                            L, n, want_lse=True)
    assert int(c.status.item()) == 0
    return c, o.cpu(), lse.cpu()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_values_that_are_not_finite_behind_a_cache(cuda_dev, d):
    rows, L = 40, 5000
    cache = ku.Cache([L], 4, 1, d, 64, seed=5)
    t, _ = pu.rows_of(rows, 4, 1, d, 1)
    c, clean, lse = chunk(cache, t, cuda_dev)
    assert chunk_workspace(c, cache, rows)[1] >= 3
    for at in (0, 130, 2600, L - 1):                          # codes of NaN: every row sees them
        page, s = cache.table[0, at // 64], at % 64
        was = cache.kv[page, 0, 1, 0, s, 3]
        cache.kv[page, 0, 1, 0, s, 3] = 127
        _, o, l = chunk(cache, t, cuda_dev)
        cache.kv[page, 0, 1, 0, s, 3] = was
        hit = torch.zeros(o.shape, dtype=torch.bool)
        hit[:, :, 3] = True
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit]) and torch.equal(l, lse)
    for at in (0, 17, rows - 1):                              # new rows, in the last part
        for what in (float("nan"), float("-inf")):
            x = t.clone()
            pu.split(x, 4, 1, d)[2][at, 0, 5] = what
            _, o, l = chunk(cache, x, cuda_dev)
            hit = torch.zeros(o.shape, dtype=torch.bool)
            hit[at:, :, 5] = True
            assert not torch.isfinite(o[hit]).any() and torch.equal(o[~hit], clean[~hit]) and torch.equal(l, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_parts_of_nothing_but_minus_infinity(cuda_dev, d):
    """Scores of -inf throughout the first parts, then throughout the later ones, against the fp64 form without them."""
    n = 2000
    assert prompt_workspace(2, 1, d, n)[1] >= 3
    g = np.random.RandomState(d)
    for lo, hi in ((0, 1500), (600, 2000), (300, 1700)):
        q, k, v = (g.standard_normal((n, h, d)) for h in (2, 1, 1))
        q[..., 3] = -1.0
        (qt, q), (kt, k), (vt, v) = ku.bf16(q), ku.bf16(k), ku.bf16(v)
        kt[lo:hi, 0, 3] = float("inf")
        from speculative_decoding_hybrid_gb300.prefill import attend_prompts
        status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
        o, lse = attend_prompts(qt.to(cuda_dev), kt.to(cuda_dev), vt.to(cuda_dev), pu.dev32([0, n], cuda_dev), n, status,
                                want_lse=True)
        assert int(status.item()) == 0
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        for r in (0, 5, lo, lo + 1, hi - 1, min(hi, n - 1), 1300, 1800, n - 2, n - 1):
            see = np.array([j for j in range(r + 1) if not lo <= j < hi], int)
            if not len(see):
                assert (o[r] == 0).all() and np.isneginf(lse[r]).all()
                continue
            x = np.stack([k[see], v[see]]).transpose(0, 2, 1, 3)
            ro, rl, ra, rw = ku.attend_request(x, q[r:r + 1], None, None, 0, pu.scale_of(d))
            ob, lb = pu.bounds(ro, rl, ra, rw, d)
            assert noted("parts of -inf: o", np.max(np.abs(o[r:r + 1] - ro) / ob)) <= 1.0, (lo, hi, r)
            assert noted("parts of -inf: lse", np.max(np.abs(lse[r:r + 1] - rl) / lb)) <= 1.0, (lo, hi, r)


@pytest.mark.parametrize("L,rows,h_q,h_kv,d,least", [(32000, 32, 16, 2, 256, 33), (14000, 5, 4, 1, 64, 17),
                                                     (30000, 20, 8, 1, 128, 33)])
def test_many_parts(cuda_dev, L, rows, h_q, h_kv, d, least):
    cache = ku.Cache([L], h_q, h_kv, d, 64, seed=2)
    t, (q, k, v) = pu.rows_of(rows, h_q, h_kv, d, 1)
    c, o, lse = chunk(cache, t, cuda_dev)
    assert chunk_workspace(c, cache, rows)[1] >= least
    x = cache.dense(0, 0)
    for a in range(0, rows, 8):                               # rows, with those before them as earlier positions
        b = min(a + 8, rows)
        y = np.concatenate([x, np.stack([k[:a], v[:a]]).transpose(0, 2, 1, 3)], 2)
        ro, rl, ra, rw = pu.attend(q[a:b], k[a:b], v[a:b], 0, ku.default_scale(d), y)
        ob, lb = pu.bounds(ro, rl, ra, rw, d)
        assert noted("many parts: o", np.max(np.abs(o[a:b].double().numpy() - ro) / ob)) <= 1.0
        assert noted("many parts: lse", np.max(np.abs(lse[a:b].double().numpy() - rl) / lb)) <= 1.0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_what_the_workspace_held_does_not_show(cuda_dev, d):
    """Sums, statistics and the units' records of parts, and the dense keys and values: the same bits over any bytes."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([5000], 4, 1, d, 64, seed=4)
    t, _ = pu.rows_of(20, 4, 1, d, 0)
    c, ref, lref = chunk(cache, t, cuda_dev)
    need, parts = chunk_workspace(c, cache, 20)
    assert parts >= 3
    q, k, v = pu.split(t.to(cuda_dev), 4, 1, d)
    table = torch.from_numpy(cache.table).to(cuda_dev)
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=cuda_dev)
        o, lse = torch.empty(20, 4, d, dtype=torch.bfloat16, device=cuda_dev), torch.empty(20, 4, device=cuda_dev)
        gs.kv8_chunk(c.c, 0, 1, 20, pu.dev32([0, 20], cuda_dev), pu.dev32([5000], cuda_dev), table, table.shape[1],
                     table.stride(0), q, q.stride(0), k, k.stride(0), v, v.stride(0), o, 4 * d, lse, 5000, 20, 5000, ws,
                     need, c.status)
        assert torch.equal(o.cpu(), ref) and torch.equal(lse.cpu(), lref)
    n = 2000
    need, parts = prompt_workspace(4, 1, d, n)
    assert parts >= 2
    t, _ = pu.rows_of(n, 4, 1, d, 0)
    ref, lref = prompt(t, 4, 1, d, cuda_dev)
    q, k, v = pu.split(t.to(cuda_dev), 4, 1, d)
    dims = gs.attn_dims(4, 1, d, 0, pu.scale_of(d))
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=cuda_dev)
        o, lse = torch.empty(n, 4, d, dtype=torch.bfloat16, device=cuda_dev), torch.empty(n, 4, device=cuda_dev)
        gs.attn_prompts(dims, 1, n, pu.dev32([0, n], cuda_dev), q, q.stride(0), k, k.stride(0), v, v.stride(0), o, 4 * d,
                        lse, n, ws, need, c.status)
        assert torch.equal(o.cpu(), ref) and torch.equal(lse.cpu(), lref)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("d,h_q", [(64, 4), (128, 4), (256, 2)])
def test_a_wait_that_runs_out_before_the_join(cuda_dev, d, h_q):
    """The join writes nothing over a record that no unit wrote."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    n = 2000
    need, parts = prompt_workspace(h_q, 1, d, n)
    assert parts >= 2
    t, _ = pu.rows_of(n, h_q, 1, d, 1)
    q, k, v = pu.split(t.to(cuda_dev), h_q, 1, d)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    o = torch.full((n, h_q, d), 7.0, dtype=torch.bfloat16, device=cuda_dev)
    ws = torch.zeros(need, dtype=torch.uint8, device=cuda_dev)
    gs.attn_selftest_prompts_timeout(gs.attn_dims(h_q, 1, d, 0, 0.1), 1, n, pu.dev32([0, n], cuda_dev), q, q.stride(0),
                                     k, k.stride(0), v, v.stride(0), o, h_q * d, n, ws, need, status, 2_000_000)
    assert int(status.item()) == gs.DEV_TIMEOUT and (o == 7.0).all()
    prompt(t, h_q, 1, d, cuda_dev)


@pytest.mark.parametrize("d,h_q", [(64, 4), (128, 4), (256, 2)])
def test_without_a_status_word(cuda_dev, d, h_q):
    """The same bits as with one, captured too; a wait that runs out writes nothing, whatever the workspace held."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    n = 2000
    need, parts = prompt_workspace(h_q, 1, d, n)
    assert parts >= 2
    t, _ = pu.rows_of(n, h_q, 1, d, 1)
    ref, lref = prompt(t, h_q, 1, d, cuda_dev)
    q, k, v = pu.split(t.to(cuda_dev), h_q, 1, d)
    cu, dims = pu.dev32([0, n], cuda_dev), gs.attn_dims(h_q, 1, d, 0, pu.scale_of(d))
    o, lse = torch.empty(n, h_q, d, dtype=torch.bfloat16, device=cuda_dev), torch.empty(n, h_q, device=cuda_dev)
    ws = torch.full((need,), 127, dtype=torch.uint8, device=cuda_dev)
    rows = (q, q.stride(0), k, k.stride(0), v, v.stride(0))

    def call():
        gs.attn_prompts(dims, 1, n, cu, *rows, o, h_q * d, lse, n, ws, need, None)
    call()
    assert torch.equal(o.cpu(), ref) and torch.equal(lse.cpu(), lref)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        call()
    for fill in (0, 255, 127):
        ws.fill_(fill)
        o.zero_()
        g.replay()
        assert torch.equal(o.cpu(), ref) and torch.equal(lse.cpu(), lref)
    ws[:] = torch.arange(need, device=cuda_dev).to(torch.uint8)
    o.fill_(7.0)
    gs.attn_selftest_prompts_timeout(dims, 1, n, cu, *rows, o, h_q * d, n, ws, need, None, 2_000_000)
    assert (o == 7.0).all()

    cache = ku.Cache([5000], h_q, 1, d, 64, seed=4)
    t = t[:20]
    c, ref, lref = chunk(cache, t, cuda_dev)
    need, parts = chunk_workspace(c, cache, 20)
    assert parts >= 2
    ws = torch.full((need,), 127, dtype=torch.uint8, device=cuda_dev)
    table = torch.from_numpy(cache.table).to(cuda_dev)
    gs.kv8_chunk(c.c, 0, 1, 20, pu.dev32([0, 20], cuda_dev), pu.dev32([5000], cuda_dev), table, table.shape[1],
                 table.stride(0), *rows, o, h_q * d, lse, 5000, 20, 5000, ws, need, None)
    assert torch.equal(o[:20].cpu(), ref) and torch.equal(lse[:20].cpu(), lref)


def test_two_calls_at_once(cuda_dev):
    """Prompts, a cut prompt and a cut chunk on three streams together: the bits of each by itself."""
    from speculative_decoding_hybrid_gb300.prefill import attend_prompts
    cache = ku.Cache([5000], 4, 1, 128, 64, seed=4)
    c = ku.gpu_cache(cache, cuda_dev)
    table, status = torch.from_numpy(cache.table).to(cuda_dev), torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    rows, calls = [], []
    for total, h_q, h_kv, d, seed in ((6000, 8, 4, 128, 1), (2000, 2, 1, 256, 2), (20, 4, 1, 128, 3)):
        rows.append(pu.split(pu.rows_of(total, h_q, h_kv, d, seed)[0].to(cuda_dev), h_q, h_kv, d))
    many, one, few, length = (pu.dev32(x, cuda_dev) for x in ([0, 2500, 2600, 6000], [0, 2000], [0, 20], [5000]))
    calls = [lambda s=None: attend_prompts(*rows[0], many, 3400, status, want_lse=True, stream=s),
             lambda s=None: attend_prompts(*rows[1], one, 2000, status, want_lse=True, stream=s),
             lambda s=None: c.attend_chunk(0, table, length, few, *rows[2], 5000, 20, want_lse=True, stream=s)]
    ref = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        got = [call(s) for call, s in zip(calls, streams)]
        torch.cuda.synchronize()
        for x, y in zip(ref, got):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert int(status.item()) == 0 and int(c.status.item()) == 0
