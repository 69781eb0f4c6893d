"""Attention over whole prompts against the fp64 form: head layouts, ragged rows, windows, work cut into parts, values
that are not finite, strides, streams, graphs and refusals."""
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


def run(rows, h_q, h_kv, d, dev, window=0, sm_scale=None, seed=0, k_scale=1.0, pad=0, edit=None, max_rows=None,
        extra=0, out=None):
    from speculative_decoding_hybrid_gb300.prefill import attend_prompts
    t, f = pu.rows_of(sum(rows) + extra, h_q, h_kv, d, seed, k_scale, pad)
    if edit:
        edit(*pu.split(t, h_q, h_kv, d))
        f = pu.split(t.double().numpy(), h_q, h_kv, d)
    q, k, v = pu.split(t.to(dev), h_q, h_kv, d)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    cu = pu.cu_of(rows)
    o, lse = attend_prompts(q, k, v, pu.dev32(cu, dev), max(rows, default=0) if max_rows is None else max_rows,
                            status, window=window, sm_scale=sm_scale, want_lse=True, out=out)
    torch.cuda.synchronize()
    return o, lse, f, cu, status


def check(name, rows, h_q, h_kv, d, dev, window=0, sm_scale=None, **kw):
    o, lse, (q, k, v), cu, status = run(rows, h_q, h_kv, d, dev, window=window, sm_scale=sm_scale, **kw)
    assert int(status.item()) == 0
    compare(name, o, lse, q, k, v, cu, window, pu.scale_of(d) if sm_scale is None else float(np.float32(sm_scale)))
    return o, lse


def compare(name, o, lse, q, k, v, cu, window, sc):
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for r, (a, b) in enumerate(zip(cu, cu[1:])):
        if a == b:
            continue
        ro, rl, ra, rw = pu.attend(q[a:b], k[a:b], v[a:b], window, sc)
        ob, lb = pu.bounds(ro, rl, ra, rw, q.shape[2])
        assert noted("prompts %s: o" % name, np.max(np.abs(o[a:b] - ro) / ob)) <= 1.0, (r, b - a)
        assert noted("prompts %s: lse" % name, np.max(np.abs(lse[a:b] - rl) / lb)) <= 1.0, (r, b - a)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (6, 2), (16, 2), (5, 5), (24, 1), (64, 1)])
def test_head_layouts(cuda_dev, d, h_q, h_kv):
    check("heads d=%d" % d, [1, 2, 0, 5, 33, 130, 0], h_q, h_kv, d, cuda_dev, seed=d + h_q)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 127, 128, 129, 255, 256, 257, 383, 513, 900])
def test_lengths(cuda_dev, d, n):
    check("lengths d=%d" % d, [n], 2, 1, d, cuda_dev, seed=n)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long(cuda_dev, d):
    check("long d=%d" % d, [2111, 70, 1500], 4, 2, d, cuda_dev, seed=d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_units_are_not_cut(cuda_dev, d):
    check("units d=%d" % d, [700] * 5, 16, 8, d, cuda_dev, seed=d)


@pytest.mark.parametrize("B", [2, 33, 128, 129, 700])
def test_many_prompts(cuda_dev, B):
    check("many prompts", [(37 * i) % 61 for i in range(B)], 4, 2, 64, cuda_dev, seed=B)


@pytest.mark.parametrize("window", [1, 2, 64, 100, 127, 128, 129, 1000])
@pytest.mark.parametrize("d", [64, 256])
def test_windows(cuda_dev, window, d):
    check("window d=%d" % d, [1, 130, 700, 1300], 4, 2, d, cuda_dev, window=window, seed=window)


@pytest.mark.parametrize("sm_scale", [-0.3, 0.0, 1.0, 1e-3])
def test_scales(cuda_dev, sm_scale):
    check("scale", [200, 3], 4, 2, 128, cuda_dev, sm_scale=sm_scale, seed=4)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_peaked(cuda_dev, d):
    """Scores of hundreds: the reference moves often, and a row is one position."""
    check("peaked d=%d" % d, [400, 150], 4, 1, d, cuda_dev, k_scale=20.0, seed=9)


def test_growing_scores(cuda_dev):
    """Every tile's scores pass the last one's by far: sums are rescaled at every tile."""
    def edit(q, k, v):
        q[:] = 1.0
        k[:] = (torch.arange(k.shape[0]) / 16.0)[:, None, None].to(torch.bfloat16)
    for d in (128, 256):
        check("growing", [900], 2, 1, d, cuda_dev, edit=edit, sm_scale=0.05)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 40])
def test_unseen_values_do_not_reach(cuda_dev, d, window):
    """NaN and infinities in the keys and values of one position reach the rows that see it and no other bit."""
    rows = [150, 300, 20]
    clean, lse, f, cu, _ = run(rows, 4, 2, d, cuda_dev, window=window, seed=3)
    for at, what in ((149, float("nan")), (150 + 131, float("inf")), (150 + 40, float("-inf")), (450, float("nan"))):
        r = np.searchsorted(cu, at, side="right") - 1

        def edit(q, k, v):
            v[at, 1, 5] = what
        o, l, _, _, status = run(rows, 4, 2, d, cuda_dev, window=window, seed=3, edit=edit)
        assert int(status.item()) == 0
        sees = torch.zeros(sum(rows), dtype=torch.bool)
        sees[at:min(int(cu[r + 1]), at + window if window else 1 << 30)] = True
        hit = torch.zeros(o.shape, dtype=torch.bool)
        hit[:, 2:, 5] = sees[:, None]                  # kv head 1 serves query heads 2 and 3
        assert not torch.isfinite(o.cpu()[hit]).any()
        assert torch.equal(o.cpu()[~hit], clean.cpu()[~hit]) and torch.equal(l, lse)
        if what == float("inf"):
            assert (o.cpu()[hit] == what).all()

        def edit(q, k, v):
            k[at, 1, 5] = float("nan")
        o, l, _, _, _ = run(rows, 4, 2, d, cuda_dev, window=window, seed=3, edit=edit)
        hit = torch.zeros(o.shape, dtype=torch.bool)
        hit[:, 2:] = sees[:, None, None]
        assert torch.isnan(o.cpu()[hit]).all() and torch.equal(o.cpu()[~hit], clean.cpu()[~hit])
        assert torch.isnan(l.cpu()[hit[..., 0]]).all() and torch.equal(l.cpu()[~hit[..., 0]], lse.cpu()[~hit[..., 0]])


def test_values_of_every_lane_are_guarded(cuda_dev):
    """Nothing of a prompt but its last row's value is finite: the other rows' outputs hold no trace of that row."""
    for d in (64, 128, 256):
        for n in (2, 128, 200):
            def edit(q, k, v):
                v[n - 1] = float("nan")
            o, _, (q, k, v), cu, _ = run([n], 2, 1, d, cuda_dev, seed=n, edit=edit)
            assert torch.isfinite(o[:n - 1]).all() and torch.isnan(o[n - 1]).all()


def test_rows_behind_the_last_prompt_stay(cuda_dev):
    for h_q, h_kv, d in ((6, 2, 128), (2, 1, 256)):
        out = torch.full((60, h_q, d), 7.0, dtype=torch.bfloat16, device=cuda_dev)
        o, lse, (q, k, v), cu, status = run([20, 0, 13], h_q, h_kv, d, cuda_dev, extra=27, out=out)
        assert int(status.item()) == 0 and (o[33:] == 7.0).all()
        compare("behind", o, lse, q, k, v, cu, 0, pu.scale_of(d))


def test_strides_and_padding(cuda_dev):
    check("padded rows", [77, 130], 6, 3, 128, cuda_dev, pad=24, seed=2)


def test_bad_rows_are_skipped(cuda_dev):
    """A request past max_rows or the rows there are is refused by itself."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    from speculative_decoding_hybrid_gb300.prefill import attend_prompts
    t, (q, k, v) = pu.rows_of(100, 4, 2, 64, 5)
    qt, kt, vt = pu.split(t.to(cuda_dev), 4, 2, 64)
    for cu, good, bound in (([30, 60, 0, 20], [(30, 60), (0, 20)], 50), ([0, 10, 90, 100], [(0, 10), (90, 100)], 50),
                            ([-5, 10, 20], [(10, 20)], 50), ([0, 40, 101], [(0, 40)], 80)):
        status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
        out = torch.full((100, 4, 64), 7.0, dtype=torch.bfloat16, device=cuda_dev)
        o, lse = attend_prompts(qt, kt, vt, pu.dev32(cu, cuda_dev), bound, status, want_lse=True, out=out)
        assert int(status.item()) == gs.DEV_ROWS_BAD
        written = torch.zeros(100, dtype=torch.bool)
        for a, b in good:
            compare("beside bad", o[a:b], lse[a:b], q[a:b], k[a:b], v[a:b], [0, b - a], 0, pu.scale_of(64))
            written[a:b] = True
        assert (o.cpu()[~written] == 7.0).all()


def test_no_rows(cuda_dev):
    for rows in ([], [0], [0, 0]):
        o, lse, _, _, status = run(rows, 4, 2, 64, cuda_dev, max_rows=5)
        assert o.shape[0] == 0 and int(status.item()) == 0


def test_same_bits_again_and_on_another_stream(cuda_dev):
    from speculative_decoding_hybrid_gb300.prefill import attend_prompts
    rows = [300, 1, 2000]
    o, lse, _, cu, _ = run(rows, 4, 1, 128, cuda_dev, seed=6)
    t, _ = pu.rows_of(sum(rows), 4, 1, 128, 6)
    q, k, v = pu.split(t.to(cuda_dev), 4, 1, 128)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o2, l2 = attend_prompts(q, k, v, pu.dev32(cu, cuda_dev), 2000, status, want_lse=True, stream=s)
        s.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_captured_and_replayed(cuda_dev):
    """A graph of two calls of different work, replayed on new rows and new lengths."""
    from speculative_decoding_hybrid_gb300.prefill import attend_prompts
    t, _ = pu.rows_of(1500, 4, 1, 128, 8)
    buf = t.to(cuda_dev)
    q, k, v = pu.split(buf, 4, 1, 128)
    cu = pu.dev32([0, 1400, 1500], cuda_dev)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    call = lambda: (attend_prompts(q, k, v, cu, 1500, status, want_lse=True),
                    attend_prompts(q, k, v, cu, 1500, status, window=99, want_lse=True))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = call()
    for seed, ends in ((8, [0, 1400, 1500]), (9, [0, 3, 1500])):
        buf.copy_(pu.rows_of(1500, 4, 1, 128, seed)[0])
        cu.copy_(pu.dev32(ends, cuda_dev))
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(out, call()):
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert int(status.item()) == 0


def test_withheld_copy_times_out(cuda_dev):
    from speculative_decoding_hybrid_gb300 import binding as gs
    for d, n in ((64, 300), (128, 300), (256, 40)):
        t, _ = pu.rows_of(n, 2, 1, d, 1)
        q, k, v = pu.split(t.to(cuda_dev), 2, 1, d)
        status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
        o = torch.full((n, 2, d), 7.0, dtype=torch.bfloat16, device=cuda_dev)
        dims = gs.attn_dims(2, 1, d, 0, 0.1)
        need = gs.attn_prompts_workspace_bytes(dims, 1, n, n)
        ws = torch.empty(max(1, need), dtype=torch.uint8, device=cuda_dev)
        gs.attn_selftest_prompts_timeout(dims, 1, n, pu.dev32([0, n], cuda_dev), q, q.stride(0), k, k.stride(0), v,
                                         v.stride(0), o, 2 * d, n, ws, need, status, 2_000_000)
        assert int(status.item()) == gs.DEV_TIMEOUT and (o == 7.0).all()
        check("after a timeout", [50], 2, 1, d, cuda_dev)


def test_arguments_are_checked(cuda_dev):
    from speculative_decoding_hybrid_gb300 import binding as gs
    from speculative_decoding_hybrid_gb300.prefill import attend_prompts
    x = lambda h, d=64, n=8, **kw: torch.zeros((n, h, d), **{**dict(dtype=torch.bfloat16, device=cuda_dev), **kw})
    cu, status = pu.dev32([0, 8], cuda_dev), pu.dev32([0], cuda_dev)
    for bad in (dict(q=x(4, dtype=torch.float16)), dict(k=x(2, n=7)), dict(v=x(1)), dict(v=x(2, d=128)),
                dict(k=x(2, device="cpu")), dict(cu_rows=cu.long()), dict(status=status.float()),
                dict(out=x(4, n=3)), dict(q=x(4).transpose(0, 1).contiguous().transpose(0, 1))):
        args = {**dict(q=x(4), k=x(2), v=x(2), cu_rows=cu, max_rows=8, status=status), **bad}
        with pytest.raises(ValueError):
            attend_prompts(**args)
    for bad, code in ((dict(q=x(3)), gs.GDN_ERR_SHAPE), (dict(q=x(4, d=96), k=x(2, d=96), v=x(2, d=96)), gs.GDN_ERR_SHAPE),
                      (dict(window=-1), gs.GDN_ERR_ARG), (dict(sm_scale=float("inf")), gs.GDN_ERR_ARG),
                      (dict(max_rows=-1), gs.GDN_ERR_ARG)):
        args = {**dict(q=x(4), k=x(2), v=x(2), cu_rows=cu, max_rows=8, status=status), **bad}
        with pytest.raises(gs.GdnError) as e:
            attend_prompts(**args)
        assert e.value.status == code
