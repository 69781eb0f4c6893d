"""Which positions a row sees, each once: weights that are powers of two and values that name their position, so that one
position left out or counted twice shows in the log-sum-exp or in a channel's output.

Heads of even number have queries of zeros (each position weighs 1: the sum is a count, exact in fp32), the others
weigh position j by 2^s_j, s_j in 0..3: one channel of q is 1, of k s_j, under a scale of ln 2.  v_j is 1 in channel
j mod d.  Error budget: scores s_j (1 + 2^-22), so weights 2^-20 of themselves, each rounded to the power of two that
it is (2^-20 more); sums and the logarithm in fp32 as in prompt_util, 2^-20 (1 + |lse|) with the weights' own; outputs
their rounding, 2^-8, and 2^-18.  A position of weight 1 of W moves lse by 1 / W: over 20 times the budget at W = 2,000,
1.4 times at 30,000; that it exceeds the budget is asserted."""
import math

import numpy as np
import pytest
import torch

import kv_util as ku
import prompt_util as pu
from gpu_util import build_lib, noted

pytestmark = pytest.mark.gpu
LN2 = float(np.float32(math.log(2.0)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def rows_of(total, h_q, h_kv, d, seed):
    g = np.random.RandomState(seed)
    q, k, v = np.zeros((total, h_q, d)), np.zeros((total, h_kv, d)), np.zeros((total, h_kv, d))
    q[:, 1::2, 7] = 1.0
    k[:, :, 7] = g.randint(0, 4, (total, h_kv))
    k[:, :, 9] = 100.0                                     # under queries of zeros
    v[np.arange(total), :, np.arange(total) % d] = 1.0
    return q, k, v


def expected(h_q, ks, vs, first, window, of=None):
    """fp64 o and lse of the rows at positions first .. end of keys' exponents ks [n, h_kv] and values vs [n, h_kv, d]."""
    n, h_kv, d = vs.shape
    o, lse = np.zeros((n - first, h_q, d)), np.zeros((n - first, h_q))
    hi = np.arange(first, n) + 1
    lo = np.maximum(0, hi - window) if window else np.zeros_like(hi)
    for h in range(h_q):
        w = 2.0 ** ks[:, h // (h_q // h_kv)] if h % 2 else np.ones(n)
        total = np.concatenate([[0.0], np.cumsum(w)])
        part = np.concatenate([np.zeros((1, d)), np.cumsum(w[:, None] * vs[:, h // (h_q // h_kv)], 0)])
        t = total[hi] - total[lo]
        o[:, h], lse[:, h] = (part[hi] - part[lo]) / t[:, None], np.log(t)
    return o, lse


def compare(name, o, lse, ro, rl, sharp=True):
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    lb = 2.0 ** -20 * (1 + rl)
    if sharp:
        assert (lb[:, ::2] < np.exp(-rl[:, ::2])).all() and (lb[:, 1::2] < np.exp(-rl[:, 1::2])).all()
    assert noted("prompt counts %s: lse" % name, np.max(np.abs(lse - rl) / lb)) <= 1.0
    assert noted("prompt counts %s: o" % name, np.max(np.abs(o - ro) / (2.0 ** -8 * ro + 2.0 ** -18))) <= 1.0


@pytest.mark.parametrize("rows,h_q,h_kv,window,cut", [
    ([1, 2, 127, 128, 129, 300, 0, 33], 4, 2, 0, None), ([513, 900], 6, 2, 0, None), ([600, 70], 64, 1, 0, None),
    ([900, 1, 1300], 4, 2, 1, None), ([900, 40], 6, 3, 100, None), ([1300, 700], 4, 2, 128, None),
    ([1300, 3], 2, 1, 129, None), ([2000], 4, 1, 1000, None), ([3000], 4, 1, 0, True), ([3000], 2, 2, 700, None),
    ([7000], 2, 1, 0, True), ([2500, 60, 700], 2, 1, 0, None), ([50 + i % 90 for i in range(150)], 2, 1, 0, None)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts(cuda_dev, d, rows, h_q, h_kv, window, cut):
    from speculative_decoding_hybrid_gb300 import binding as gs
    from speculative_decoding_hybrid_gb300.prefill import attend_prompts
    R = sum(rows)
    q, k, v = rows_of(R, h_q, h_kv, d, R)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    if cut:
        assert gs.attn_prompts_workspace_bytes(gs.attn_dims(h_q, h_kv, d, window, LN2), len(rows), R, max(rows)) > 0
    o, lse = attend_prompts(*(ku.bf16(x)[0].to(cuda_dev) for x in (q, k, v)), pu.dev32(pu.cu_of(rows), cuda_dev),
                            max(rows), status, window=window, sm_scale=LN2, want_lse=True)
    assert int(status.item()) == 0
    cu = pu.cu_of(rows)
    for a, b in zip(cu, cu[1:]):
        if a < b:
            compare("prompts d=%d" % d, o[a:b], lse[a:b], *expected(h_q, k[a:b, :, 7], v[a:b], 0, window))


@pytest.mark.parametrize("lens,rows,h_q,h_kv,T,window", [
    ([5000, 130, 2500, 0], [20, 17, 33, 140], 4, 1, 64, 0), ([9000], [3], 4, 1, 16, 0), ([9000, 40], [300, 9], 2, 1, 128, 0),
    ([777, 2000, 3], [700, 40, 129], 6, 2, 32, 100), ([5000, 700], [40, 300], 2, 1, 16, 1000),
    ([100 + i % 40 for i in range(140)], [1 + i % 50 for i in range(140)], 2, 1, 32, 0), ([32000], [32], 4, 2, 64, 0)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_chunks(cuda_dev, d, lens, rows, h_q, h_kv, T, window):
    R = sum(rows)
    cache = ku.Cache(lens, h_q, h_kv, d, T, seed=R)
    g = np.random.RandomState(R)
    cache.scale[:] = 1.0
    cache.kv[:] = 0
    cache.kv[:, 0, 0, :, :, 7] = ku.encode(g.randint(0, 4, cache.kv[:, 0, 0, :, :, 7].shape).astype(float))
    for r, n in enumerate(lens):
        t = np.arange(n)
        cache.kv[cache.table[r, t // T], 0, 1, :, t % T, t % d] = ku.encode(1.0)
    q, k, v = rows_of(R, h_q, h_kv, d, R)
    c = ku.gpu_cache(cache, cuda_dev, window, LN2)
    o, lse = c.attend_chunk(0, torch.from_numpy(cache.table).to(cuda_dev), pu.dev32(lens, cuda_dev),
                            pu.dev32(pu.cu_of(rows), cuda_dev), *(ku.bf16(x)[0].to(cuda_dev) for x in (q, k, v)),
                            max(lens), max(rows), sum(lens), want_lse=True)
    assert int(c.status.item()) == 0
    cu = pu.cu_of(rows)
    for r, (a, b) in enumerate(zip(cu, cu[1:])):
        x = cache.dense(r, 0).transpose(0, 2, 1, 3)            # [2, length, h_kv, d]
        ks, vs = np.concatenate([x[0, :, :, 7], k[a:b, :, 7]]), np.concatenate([x[1], v[a:b]])
        compare("chunks d=%d" % d, o[a:b], lse[a:b], *expected(h_q, ks, vs, lens[r], window), sharp=lens[r] < 10000)
