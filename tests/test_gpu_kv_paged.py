"""The paged cache as it is used: prompts, forks, verification transactions
beside GatedDeltaNet layers, commits of the accepted rows, requests that leave
and compaction, followed request by request against the fp64 forms."""
import os
import sys

import numpy as np
import pytest
import torch

import kv_util as ku
from gpu_util import build_lib, noted

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))


class Follow:
    """What each request's cache should hold, layer by layer: its committed rows, appended as they were."""

    def __init__(self, kv, requests):
        self.h, self.d, self.T, self.layers = kv.h_kv, kv.d, kv.page_tokens, kv.kv.shape[1]
        cap = kv.tables.shape[1] * self.T
        self.c = [ku.Cache([0], kv.h_q, self.h, self.d, self.T, layers=self.layers, room=[cap], seed=r)
                  for r in range(requests)]

    def append(self, r, rows):
        n = 0
        for layer, (k, v) in enumerate(rows):
            n = k.shape[0]
            ku.append_request(self.c[r], 0, layer, k.double().cpu().numpy(), v.double().cpu().numpy())
        self.c[r].lens[0] += n

    def fork(self, src, dst, n):
        a, b = self.c[src], self.c[dst]
        for j in range(-(-n // self.T)):
            b.kv[b.table[0, j]], b.scale[b.table[0, j]] = a.kv[a.table[0, j]], a.scale[a.table[0, j]]
        b.lens[0] = n

    def check(self, kv, r):
        """Every stored value of request r, bit for bit."""
        n = int(kv.length[r])
        assert n == self.c[r].lens[0]
        ids = torch.from_numpy(kv.tables[r, :-(-n // self.T)].astype(np.int64)).to(kv.kv.device)
        codes, scale = kv.kv[ids].cpu().numpy(), kv.scale[ids].cpu().numpy().astype(np.float64)
        for layer in range(self.layers):
            x = ku.VALUES[codes[:, layer]] * scale[:, layer].swapaxes(1, 2)[..., None, None]
            got = x.transpose(1, 2, 0, 3, 4).reshape(2, self.h, -1, self.d)[:, :, :n]
            assert np.array_equal(got, self.c[r].dense(0, layer, n)), (r, layer)

    def attend(self, name, r, seen, a, b, o_all):
        for layer, (q, k, v, o) in enumerate(seen):
            q, k, v = (t[a:b].double().cpu().numpy() for t in (q, k, v))
            ro, rl, ra, rw = ku.attend_request(self.c[r].dense(0, layer), q, k, v, 0, ku.default_scale(self.d))
            ob, _ = ku.attend_bounds(ro, rl, ra, rw, self.d)
            got = o_all[layer][a:b].double().cpu().numpy()
            assert noted(name, np.max(np.abs(got - ro) / ob)) <= 1.0, (r, layer)


@pytest.mark.parametrize("d,page_tokens,h_q,h_kv", [(128, 32, 8, 2), (256, 64, 16, 2), (64, 16, 6, 6)])
def test_transactions_of_a_hybrid(cuda_dev, d, page_tokens, h_q, h_kv):
    import hybrid_decode as hd
    B, prompt = 4, 150
    h = hd.HybridDecode(B, 2, 2, 400, h_q=h_q, h_kv=h_kv, d=d, page_tokens=page_tokens, seed=d)
    f = Follow(h.kv, B)
    f.append(0, h.prompt(0, prompt))
    f.check(h.kv, 0)
    for r in range(1, B):
        h.kv.fork(0, r, prompt - 7 * (r - 1))
        f.fork(0, r, prompt - 7 * (r - 1))
    g = np.random.RandomState(d)
    for step in range(10):
        drafts = [int(x) for x in g.randint(0, 4, B)]
        before = [int(x) for x in h.kv.length]
        seen, accept = h.step(drafts)
        a = 0
        for r in range(B):
            b = a + drafts[r] + 1
            f.attend("kv transactions d=%d: o" % d, r, seen, a, b, [x[3] for x in seen])
            n = int(accept[r]) + 1
            f.append(r, [(k[a:a + n], v[a:a + n]) for _, k, v, _ in seen])
            assert int(h.kv.length[r]) == before[r] + n
            a = b
        if step in (3, 7):
            for r in range(B):
                f.check(h.kv, r)
        if step == 4:
            h.kv.free(2)
            h.kv.fork(0, 2, 100)
            f.fork(0, 2, 100)
            assert h.kv.compact() > 0
            live = len(set(h.kv.tables[h.kv.tables >= 0].tolist()))
            assert h.kv.tables.max() < live
            for r in range(B):
                f.check(h.kv, r)


def test_a_refused_request_commits_nothing(cuda_dev):
    """An accept length of -1 (the greedy acceptance refused the rows) leaves the request's pages as they were."""
    import hybrid_decode as hd
    h = hd.HybridDecode(2, 1, 1, 200, seed=5)
    for r in range(2):
        h.prompt(r, 50)
    kv = h.kv
    kv.reserve([0, 1], [4, 4])
    table, length = kv.upload([0, 1])
    before = kv.kv.clone()
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device=cuda_dev)
    _, k, v = h.attention_rows(8)
    kv.append(0, table, length, cu, k, v, accept_len=torch.tensor([-1, 2], dtype=torch.int32, device=cuda_dev))
    pages = torch.from_numpy(kv.tables[0, :kv.n_pages[0]].astype(np.int64)).to(cuda_dev)
    assert torch.equal(kv.kv[pages], before[pages]) and not torch.equal(kv.kv, before)
    assert int(kv.status.item()) == 0


def test_uploads_do_not_overtake_each_other(cuda_dev):
    """Tables uploaded back to back: each call reads its own."""
    import hybrid_decode as hd
    h = hd.HybridDecode(3, 1, 1, 300, seed=6)
    rows = [h.prompt(r, n) for r, n in enumerate((40, 200, 120))]
    assert len(rows) == 3
    q, k, v = h.attention_rows(2)
    cu = torch.tensor([0, 2], dtype=torch.int32, device=cuda_dev)
    outs = []
    for r in (0, 1, 2, 1, 0):
        table, length = h.kv.upload([r])
        outs.append(h.kv.attend(0, table, length, cu, q, k, v, max_len=300, max_rows=2, split_tokens=256)[0])
    assert torch.equal(outs[0], outs[4]) and torch.equal(outs[1], outs[3]) and not torch.equal(outs[0], outs[1])


def test_the_example_runs(cuda_dev, capsys):
    import hybrid_decode as hd
    h = hd.main(["--requests", "3", "--prompt", "100", "--steps", "6", "--layers", "2", "--attention", "1"])
    assert h.accepted > 0 and "drafts accepted" in capsys.readouterr().out
