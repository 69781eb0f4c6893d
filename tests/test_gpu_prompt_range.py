"""Attention of prompts and chunks where scores and values are far from ordinary: finite scores up to 2^125 that are not
powers of two, infinite ones, rows that see nothing but -inf, values up to 2^90, scales of next to nothing, in whole
units and in units cut into parts; against the fp64 form.

Scores come of one channel of q and of k, so that the products of their 8-bit significands are exact in fp32 and a
score's error is the scale's alone: the budget is prompt_util's without its term for scores.  Weights of positions whose
scores differ by z sm_scale (in powers of two) are then off by 2^-23 z, below 2^-15 as far as they count."""
import math

import numpy as np
import pytest
import torch

import kv_util as ku
import prompt_util as pu
from gpu_util import build_lib, noted

pytestmark = pytest.mark.gpu
WEIGHTS = 2.0 ** -15


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def prompts(rows, q, k, v, dev, window=0, sm_scale=None, cut=None):
    from speculative_decoding_hybrid_gb300 import binding as gs
    from speculative_decoding_hybrid_gb300.prefill import attend_prompts
    (qt, q), (kt, k), (vt, v) = ku.bf16(q), ku.bf16(k), ku.bf16(v)
    d, n = q.shape[2], sum(rows)
    if cut is not None:
        need = gs.attn_prompts_workspace_bytes(gs.attn_dims(q.shape[1], k.shape[1], d, window, 0.1), len(rows), n, max(rows))
        assert (need > 0) == cut
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    o, lse = attend_prompts(qt.to(dev), kt.to(dev), vt.to(dev), pu.dev32(pu.cu_of(rows), dev), max(rows), status,
                            window=window, sm_scale=sm_scale, want_lse=True)
    assert int(status.item()) == 0
    return (o.double().cpu().numpy(), lse.double().cpu().numpy()), (q, k, v)


def chunk(cache, rows, q, k, v, dev, sm_scale=None):
    """One request's rows behind its cache; the work is cut."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    (qt, q), (kt, k), (vt, v) = ku.bf16(q), ku.bf16(k), ku.bf16(v)
    L, (h_kv, d) = cache.lens[0], k.shape[1:]
    c = ku.gpu_cache(cache, dev, 0, sm_scale)
    assert gs.kv8_chunk_workspace_bytes(c.c, 1, rows, L, rows, L) > (L + rows) * h_kv * d * 4
    o, lse = c.attend_chunk(0, torch.from_numpy(cache.table).to(dev), pu.dev32([L], dev), pu.dev32([0, rows], dev),
                            qt.to(dev), kt.to(dev), vt.to(dev), L, rows, want_lse=True)
    assert int(c.status.item()) == 0
    return (o.double().cpu().numpy(), lse.double().cpu().numpy()), (q, k, v)


def check(name, got, ref):
    """ref: what prompt_util.attend gives; scores without an error of their own."""
    (o, lse), (ro, rl, ra, _) = got, ref
    ob, lb = pu.bounds(ro, rl, ra, np.zeros(rl.shape), o.shape[2])
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), none) and (o[none] == 0).all()
    assert np.isfinite(o).all() and np.isfinite(lse[~none]).all()
    assert noted("prompt range %s: o" % name, np.max(np.abs(o - ro) / (ob + WEIGHTS * ra))) <= 1.0
    assert noted("prompt range %s: lse" % name, np.max(np.abs(lse - rl)[~none] / (lb + WEIGHTS)[~none], initial=0.0)) <= 1.0


# What the keys' one channel holds, position by position, as a multiple of the score's size: all of one score, scores
# that pass one another tile by tile and inside tiles, ones that fall, ones that run from -1 through 0 to 1 in both
# scales, and small ones before large ones (the reference passes from the one kind to the other and back).
def _keys(kind, n):
    t = np.arange(n)
    if kind == "one":
        return np.full(n, 1.7)
    if kind == "least":
        return np.full(n, -1.7)
    if kind == "rising":
        return 1.0 + (t * 7 % 128) / 128.0 + 0.25 * (t // 64)
    if kind == "falling":
        return 1.0 - 1.9 * t / n
    if kind == "toward zero":
        return -1.7 * 2.0 ** -(t / 4.0)
    if kind == "away from zero":
        return 1.7 * 2.0 ** ((t - n) / 3.0)
    if kind == "both":
        return np.where(t % 50 < 25, -1.0, 1.0) * 1.3 * 2.0 ** (-((t * 37) % 90) / 2.0)
    raise ValueError(kind)


KINDS = ["one", "least", "rising", "falling", "toward zero", "away from zero", "both"]
SIZES = [8, 16, 19, 20, 21, 23, 26, 33, 36, 40, 60, 90, 122]


def _scores(n, h_q, h_kv, d, kind, e, seed):
    """Rows whose scores before the scale are about +-2^e (heads: 2^e, its negative, 2^(e/2) and 1.1 times it)."""
    g = np.random.RandomState(seed)
    q, k = np.zeros((n, h_q, d)), np.zeros((n, h_kv, d))
    at = 5 * seed % d
    a = e // 2
    for h in range(h_q):
        q[:, h, at] = (1.3 * 2.0 ** (e - a), -1.3 * 2.0 ** (e - a), 1.6 * 2.0 ** (e // 2 - a), 1.1 * 2.0 ** (e - a))[h % 4]
    k[:, :, at] = (_keys(kind, n) * 2.0 ** a)[:, None]
    return q, k, g.standard_normal((n, h_kv, d))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_of_any_size(cuda_dev, d, kind):
    sc = pu.scale_of(d)
    for e in SIZES:
        rows = [1, 37, 300]
        parts = [_scores(n, 4, 1, d, kind, e, e + n) for n in rows]
        got, (q, k, v) = prompts(rows, *(np.concatenate(x) for x in zip(*parts)), cuda_dev, cut=False)
        cu = pu.cu_of(rows)
        for a, b in zip(cu, cu[1:]):
            check("scores d=%d" % d, tuple(x[a:b] for x in got), pu.attend(q[a:b], k[a:b], v[a:b], 0, sc))


@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("e", [10, 21, 36, 60, 120])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_of_any_size_in_parts(cuda_dev, d, e, window):
    n = 1500
    for kind in ("one", "rising", "toward zero", "away from zero", "both") if not window else ("both",):
        q, k, v = _scores(n, 2, 1, d, kind, e, 3)
        got, (q, k, v) = prompts([n], q, k, v, cuda_dev, window, cut=not window)
        for a, b in ((0, 20), (700, 720), (n - 40, n)):       # rows, with those before them as earlier positions
            x = np.stack([k[:a], v[:a]]).transpose(0, 2, 1, 3)
            check("parts d=%d" % d, tuple(y[a:b] for y in got),
                  pu.attend(q[a:b], k[a:b], v[a:b], window, pu.scale_of(d), x))


@pytest.mark.parametrize("e", [12, 22, 36, 60, 110])
@pytest.mark.parametrize("d,L", [(64, 5000), (128, 5000), (256, 5000), (128, 13000)])
def test_scores_of_any_size_behind_a_cache(cuda_dev, d, L, e):
    """The cache's keys: one channel, a score's sizes page by page, alike within most pages."""
    rows = 20
    for flip in (1.0, -1.0):
        cache = ku.Cache([L], 4, 1, d, 64, seed=e)
        q, k, v = _scores(rows, 4, 1, d, "rising", e, 1)
        at = 5 % d
        cache.kv[:, 0, 0] = 0
        cache.kv[:, 0, 0, :, :, at] = ku.encode(flip * 416.0)
        cache.kv[cache.table[0, 3], 0, 0, :, 5:9, at] = ku.encode(np.array([448.0, 448.0, 1.0, -352.0]))
        for j in range(cache.table.shape[1]):
            cache.scale[cache.table[0, j], 0, :, 0] = 2.0 ** (e // 2 - 8 - (j * 13 % 29 if j % 5 else 0))
        got, (q, k, v) = chunk(cache, rows, q, k, v, cuda_dev)
        check("cache d=%d" % d, got, pu.attend(q, k, v, 0, pu.scale_of(d), cache.dense(0, 0)))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [200, 1500])
def test_scores_of_minus_infinity_have_no_weight(cuda_dev, d, n):
    """Infinite keys under a head of positive queries (its rows are NaN) and one of negative ones (no weight there)."""
    sc = pu.scale_of(d)
    g = np.random.RandomState(d)
    q, k, v = (g.standard_normal((n, h, d)) for h in (2, 1, 1))
    q[:, 0, 3], q[:, 1, 3] = 1.0, -1.0
    for seen in (range(0, n), range(0, 5), range(100, 180), range(3, n, 2), range(0, n - 1), range(n - 1, n)):
        seen = list(seen)
        kk = k.copy()
        kk[seen, 0, 3] = np.inf
        (o, lse), (q64, k64, v64) = prompts([n], q, kk, v, cuda_dev, cut=n > 1000)
        first = np.arange(n) >= seen[0]
        assert np.isnan(o[first, 0]).all() and np.isnan(lse[first, 0]).all()
        gone = np.zeros(n, bool)
        gone[seen] = True
        k64[gone] = 0.0
        s = np.einsum("nd,td->nt", q64[:, 1], k64[:, 0]) * sc
        s[:, gone] = -np.inf
        s = np.where(np.tri(n, dtype=bool), s, -np.inf)
        top = s.max(1, keepdims=True)
        p = np.exp(s - np.where(np.isinf(top), 0.0, top))
        total = p.sum(1, keepdims=True)
        with np.errstate(divide="ignore"):
            rl = np.log(total[:, 0]) + np.where(np.isinf(top), 0.0, top)[:, 0]
        p /= np.where(total > 0, total, 1.0)
        worst = np.where(np.tri(n, dtype=bool), np.abs(q64[:, 1]) @ np.abs(k64[:, 0]).T, 0.0).max(1) * sc
        ro, ra = p @ v64[:, 0], p @ np.abs(v64[:, 0])
        ob, lb = pu.bounds(ro, rl, ra, worst, d)
        none = np.isneginf(rl)
        assert (o[none, 1] == 0).all() and np.array_equal(np.isneginf(lse[:, 1]), none)
        assert noted("prompt range -inf: o", np.max(np.abs(o[:, 1] - ro) / ob)) <= 1.0
        assert noted("prompt range -inf: lse", np.max(np.abs(lse[:, 1] - rl)[~none] / lb[~none], initial=0.0)) <= 1.0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_values(cuda_dev, d):
    """|v| up to 2^90, with a reference that lags its rows' largest score."""
    for n, cut in ((300, False), (1500, True)):
        g = np.random.RandomState(n)
        q, k, v = (g.standard_normal((n, h, d)) for h in (2, 1, 1))
        q[..., 0], k[..., 0] = 1.0, np.linspace(0, 60, n)[:, None]
        v = np.clip(v * 2.0 ** 89, -2.0 ** 90, 2.0 ** 90)
        (o, lse), (q, k, v) = prompts([n], q, k, v, cuda_dev, sm_scale=1.0 if d == 64 else 0.1, cut=cut)
        ro, rl, ra, rw = pu.attend(q, k, v, 0, 1.0 if d == 64 else float(np.float32(0.1)))
        ob, lb = pu.bounds(ro, rl, ra, rw, d)
        assert noted("prompt range 2^90: o", np.max(np.abs(o - ro) / ob)) <= 1.0
        assert noted("prompt range 2^90: lse", np.max(np.abs(lse - rl) / lb)) <= 1.0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("n", [200, 1500])
def test_rows_of_nothing_but_minus_infinity_are_zero(cuda_dev, d, what, n):
    """o = 0 and lse = -inf whatever the values hold there, in tiles that every row sees and in others."""
    q, k, v = np.zeros((n, 1, d)), np.zeros((n, 1, d)), np.random.RandomState(d).standard_normal((n, 1, d))
    q[:, 0, 3], k[:, 0, 3] = -1.0, np.inf
    k[n - 1, 0, 3] = 1.0
    v[[0, 50, 127, 128, 150, n - 2], 0, 5] = what
    (o, lse), _ = prompts([n], q, k, v, cuda_dev, cut=n > 1000)
    assert (o[:n - 1] == 0).all() and np.isneginf(lse[:n - 1]).all()
    assert np.isfinite(lse[n - 1]).all() and np.isfinite(np.delete(o[n - 1, 0], 5)).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sm_scale", [0.0, 1e-42, -1e-42, 1e-39, -2e-38])
def test_scales_of_next_to_nothing(cuda_dev, d, sm_scale):
    """Large q.k under a scale of zero, or of a subnormal number: nearly every position weighs the same."""
    for n, cut in ((150, False), (1500, True)):
        q, k, v = _scores(n, 2, 1, d, "both", 122, 3)
        got, (q, k, v) = prompts([n], q, k, v, cuda_dev, sm_scale=sm_scale, cut=cut)
        check("small scale", got, pu.attend(q, k, v, 0, float(np.float32(sm_scale))))


def test_the_log_of_a_sum_near_one(cuda_dev):
    """Rows of two positions, scores 0 and -s: lse = log(1 + e^-s), to 2^-22.  (The smaller weight is off by 2^-22.5 of
    itself, their sum by 2^-24 of itself, its logarithm to base 2 and the product with ln 2 by 2^-24 each: 2^-22.2.)"""
    s = np.concatenate([np.arange(0, 256) / 256.0 * 2.0 ** e for e in range(5)])
    s = ku.bf16(s)[1]
    for d in (64, 128, 256):
        n = len(s)
        q, k, v = np.zeros((2 * n, 1, d)), np.zeros((2 * n, 1, d)), np.zeros((2 * n, 1, d))
        q[..., 3] = -1.0
        k[1::2, 0, 3] = s
        (_, lse), _ = prompts([2] * n, q, k, v, cuda_dev, sm_scale=1.0)
        assert (lse[::2] == 0).all()
        assert noted("prompt range log: lse", np.max(np.abs(lse[1::2, 0] - np.log1p(np.exp(-s)))) * 2.0 ** 22) <= 1.0


def test_a_scale_in_a_tensor_is_read_at_every_call(cuda_dev):
    q, k, v = (np.random.RandomState(1).standard_normal((40, h, 64)) for h in (2, 1, 1))
    scale = torch.tensor(0.125)
    for x in (0.125, 0.5, -0.25):
        scale.fill_(x)
        (o, lse), _ = prompts([40], q, k, v, cuda_dev, sm_scale=scale)
        (ro, rl), _ = prompts([40], q, k, v, cuda_dev, sm_scale=x)
        assert np.array_equal(o, ro) and np.array_equal(lse, rl)
