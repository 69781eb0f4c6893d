"""Rotary positions against the fp64 form: layouts, parts of a head, far positions, scalings, in place, refusals."""
import math

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


def turned(x, pos, f, m, rot, inter):
    """fp64 rows x [n, h, d] at positions pos, channel pair by channel pair."""
    y = x.copy()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if inter else (j, j + rot // 2)
        c, s = m * np.cos(pos * f[j])[:, None], m * np.sin(pos * f[j])[:, None]
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, a] * s + x[:, :, b] * c
    return y


# Error budget of a pair's outputs with r = magnitude * hypot(a, b): half a bf16 step, 2^-8 of the value; the angle,
# 2^-33 of a turn from the table's rounding and 2^-24 of half a turn from fp32's: below 2^-21 r; the oracle's own
# angle, position * f in fp64, 2^-52 of it: below 2^-30 for angles up to 2^21; cosine, sine, two products and a sum in
# fp32: 2^-21 r together.
def check(name, dev, rows, lens, h_q, h_kv, d, rot, inter=False, seed=0, in_place=False, pad=0, extra=0, **kw):
    from speculative_decoding_hybrid_gb300.prefill import Rope
    R = sum(rows)
    t, _ = pu.rows_of(R + extra, h_q, h_kv, d, seed, pad=pad)
    q64, k64, _ = pu.split(t.double().numpy(), h_q, h_kv, d)
    q, k, v = pu.split(t.to(dev), h_q, h_kv, d)
    rope = Rope(d, rot, interleaved=inter, device=dev, **kw)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    lens_t = None if lens is None else pu.dev32(lens, dev)
    qo, ko = rope.rotate(q, k, pu.dev32(pu.cu_of(rows), dev), lens_t, status, in_place=in_place)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    if in_place:
        assert qo is q and ko is k and torch.equal(v.cpu(), pu.split(t, h_q, h_kv, d)[2])
    pos = np.concatenate([[(0 if lens is None else lens[r]) + np.arange(n)] for r, n in enumerate(rows)], 1)[0] \
        if len(rows) == 1 else np.concatenate([(0 if lens is None else lens[r]) + np.arange(n) for r, n in enumerate(rows)])
    for x, y in ((q64, qo), (k64, ko)):
        ref = turned(x[:R], pos.astype(np.float64), rope.frequencies, rope.magnitude, rot, inter)
        z = x[:R, :, :rot]
        r = np.hypot(z[..., 0::2], z[..., 1::2]) if inter else np.hypot(z[..., :rot // 2], z[..., rot // 2:])
        r = rope.magnitude * (np.repeat(r, 2, -1) if inter else np.concatenate([r, r], -1))
        bound = 2.0 ** -8 * np.abs(ref[..., :rot]) + (2.0 ** -20 + 2.0 ** -30) * r + 1e-30
        got = y.double().cpu().numpy()[:R]
        assert noted("rope %s" % name, np.max(np.abs(got[..., :rot] - ref[..., :rot]) / bound, initial=0.0)) <= 1.0
        assert np.array_equal(got[..., rot:], x[:R, :, rot:])
    return qo, ko


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 38), (64, 2), (128, 128), (128, 64), (128, 70), (256, 64),
                                   (256, 256), (256, 134), (8, 8), (80, 48), (512, 512), (96, 96)])
def test_layouts(cuda_dev, inter, d, rot):
    check("layouts", cuda_dev, [3, 1, 0, 40, 300], [0, 5, 9, 1000, 77], 6, 2, d, rot, inter, seed=rot)


@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (16, 2), (5, 5), (64, 1), (40, 8)])
@pytest.mark.parametrize("inter", [False, True])
def test_heads(cuda_dev, h_q, h_kv, inter):
    check("heads", cuda_dev, [9, 2], [0, 3], h_q, h_kv, 128, 96, inter)


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions(cuda_dev, inter):
    lens = [0, 4095, 131071, 1000000, (1 << 21) - 7, 262144, 999983]
    check("far", cuda_dev, [2] * len(lens), lens, 4, 2, 128, 128, inter, base=1e6)


def test_the_farthest_position(cuda_dev):
    """2^31 - 1, against an angle reduced in integers."""
    from speculative_decoding_hybrid_gb300.prefill import Rope
    rope = Rope(64, device=cuda_dev)
    t, (q64, k64, _) = pu.rows_of(2, 1, 1, 64, 3)
    q, k, _ = pu.split(t.to(cuda_dev), 1, 1, 64)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    qo, _ = rope.rotate(q, k, pu.dev32([0, 2], cuda_dev), pu.dev32([(1 << 31) - 3], cuda_dev), status)
    assert int(status.item()) == 0
    for i, p in enumerate(((1 << 31) - 3, (1 << 31) - 2)):
        for j, n in enumerate(rope.turns.cpu().numpy().view(np.uint64).tolist()):
            th = 2 * math.pi * ((p * n) % (1 << 64)) / 2.0 ** 64
            a, b = q64[i, 0, j], q64[i, 0, j + 32]
            for got, ref in ((qo[i, 0, j], a * math.cos(th) - b * math.sin(th)),
                             (qo[i, 0, j + 32], a * math.sin(th) + b * math.cos(th))):
                assert abs(float(got) - ref) <= 2.0 ** -8 * abs(ref) + 2.0 ** -20 * math.hypot(a, b)


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                                dict(scaling="parts", factor=32.0, trained=4096, base=5e5), dict(base=100.0)])
def test_scalings(cuda_dev, kw):
    check("scalings", cuda_dev, [50, 7], [8000, 120000], 4, 4, 128, 128, **kw)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [128, 48, 38])
def test_in_place(cuda_dev, inter, rot):
    qo, _ = check("in place", cuda_dev, [33, 100], [5, 0], 8, 2, 128, rot, inter, seed=1, in_place=True, pad=16)
    q2, _ = check("not in place", cuda_dev, [33, 100], [5, 0], 8, 2, 128, rot, inter, seed=1, pad=16)
    assert torch.equal(qo, q2)


def test_many_rows_and_one(cuda_dev):
    """Every way of dealing rows to threads gives a row the same bits."""
    whole, _ = check("many", cuda_dev, [5000], None, 4, 2, 64, 32, seed=2)
    t, _ = pu.rows_of(5000, 4, 2, 64, 2)
    from speculative_decoding_hybrid_gb300.prefill import Rope
    rope = Rope(64, 32, device=cuda_dev)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    q, k, _ = pu.split(t.to(cuda_dev), 4, 2, 64)
    for a, n in ((0, 1), (4000, 1), (77, 40), (1000, 1500)):
        qo, ko = rope.rotate(q[a:a + n], k[a:a + n], pu.dev32([0, n], cuda_dev), pu.dev32([a], cuda_dev), status)
        assert torch.equal(qo, whole[a:a + n])
        only, none = rope.rotate(q[a:a + n], None, pu.dev32([0, n], cuda_dev), pu.dev32([a], cuda_dev), status)
        assert none is None and torch.equal(only, qo)


def test_many_requests(cuda_dev):
    rows = [1, 0, 2] * 700
    check("many requests", cuda_dev, rows, list(range(len(rows))), 2, 1, 64, 64)


def test_what_is_not_finite_stays_in_its_pair(cuda_dev):
    from speculative_decoding_hybrid_gb300.prefill import Rope
    t, _ = pu.rows_of(4, 2, 1, 64, 4)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    cu = pu.dev32([0, 4], cuda_dev)
    for inter, mate in ((False, 5 + 32), (True, 4)):
        rope = Rope(64, interleaved=inter, device=cuda_dev)
        q, k, _ = pu.split(t.to(cuda_dev), 2, 1, 64)
        clean, _ = rope.rotate(q, k, cu, None, status)
        q = q.clone()
        q[1, 0, 5] = float("nan")
        got, _ = rope.rotate(q, k, cu, None, status)
        hit = torch.zeros(got.shape, dtype=torch.bool, device=cuda_dev)
        hit[1, 0, 5] = hit[1, 0, mate] = True
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


def test_bad_rows_and_rows_of_nobody(cuda_dev):
    from speculative_decoding_hybrid_gb300 import binding as gs
    from speculative_decoding_hybrid_gb300.prefill import Rope
    rope = Rope(64, device=cuda_dev)
    t, _ = pu.rows_of(40, 2, 1, 64, 4)
    q, k, _ = pu.split(t.to(cuda_dev), 2, 1, 64)
    for cu, lens, bad, good in (([0, 10, 41], [0, 0], True, (0, 10)), ([0, 10, 20], [-1, 3], True, (10, 20)),
                                ([0, 10, 20], [3, (1 << 31) - 5], True, (0, 10)), ([5, 5, 9], [1, 2], False, (5, 9)),
                                ([-3, 4, 12], [0, 0], True, (4, 12))):
        status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
        out = torch.full((40, 2, 64), 7.0, dtype=torch.bfloat16, device=cuda_dev)
        rope.rotate(q, k, pu.dev32(cu, cuda_dev), pu.dev32(lens, cuda_dev), status, q_out=out)
        assert int(status.item()) == (gs.DEV_ROWS_BAD if bad else 0)
        a, b = good
        assert not (out[a:b] == 7.0).all(-1).any() and (out[:a] == 7.0).all() and (out[b:] == 7.0).all()


def test_streams_and_graphs(cuda_dev):
    from speculative_decoding_hybrid_gb300.prefill import Rope
    rope = Rope(128, 64, device=cuda_dev)
    t, _ = pu.rows_of(300, 8, 2, 128, 4)
    buf = t.to(cuda_dev)
    q, k, _ = pu.split(buf, 8, 2, 128)
    cu, lens = pu.dev32([0, 100, 300], cuda_dev), pu.dev32([7, 9000], cuda_dev)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    ref = rope.rotate(q, k, cu, lens, status)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = rope.rotate(q, k, cu, lens, status, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = rope.rotate(q, k, cu, lens, status)
    lens.copy_(pu.dev32([123456, 3], cuda_dev))
    g.replay()
    ref = rope.rotate(q, k, cu, lens, status)
    torch.cuda.synchronize()
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


def test_arguments_are_checked(cuda_dev):
    from speculative_decoding_hybrid_gb300.prefill import Rope
    rope = Rope(64, device=cuda_dev)
    x = lambda h, n=8, d=64, **kw: torch.zeros((n, h, d), **{**dict(dtype=torch.bfloat16, device=cuda_dev), **kw})
    cu, status = pu.dev32([0, 8], cuda_dev), pu.dev32([0], cuda_dev)
    for bad in (dict(q=x(4, dtype=torch.float32)), dict(q=x(4, d=128)), dict(k=x(2, n=7)), dict(k=x(2, device="cpu")),
                dict(cu_rows=cu.long()), dict(cache_len=pu.dev32([], cuda_dev)), dict(status=status.float()),
                dict(q_out=x(3)), dict(in_place=True, q_out=x(4)), dict(k=None, k_out=x(2)),
                dict(q=x(4).transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            rope.rotate(**{**dict(q=x(4), k=x(2), cu_rows=cu, cache_len=None, status=status), **bad})
