"""The paged 8-bit cache's calls at their smallest: no rows at all, one row or one head of any stride."""
import numpy as np
import pytest
import torch

import kv_util as ku
from gpu_util import build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def ints(dev, *x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("split", [0, 128])
def test_no_rows_in_the_whole_batch(cuda_dev, d, split):
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([2000, 3, 0], 8, 2, d, 64, seed=d)
    c = ku.gpu_cache(cache, cuda_dev)
    table, lens = torch.from_numpy(cache.table).to(cuda_dev), ints(cuda_dev, *cache.lens)
    q = torch.empty((0, 8, d), dtype=torch.bfloat16, device=cuda_dev)
    k = torch.empty((0, 2, d), dtype=torch.bfloat16, device=cuda_dev)
    kv, scale = c.kv.clone(), c.scale.clone()
    cu = ints(cuda_dev, 0, 0, 0, 0)
    for new in ((k, k), (None, None)):
        o, lse = c.attend(0, table, lens, cu, q, *new, max_len=2000, split_tokens=split, want_lse=True)
        assert o.shape == (0, 8, d) and lse.shape == (0, 8)
    c.append(0, table, lens, cu, k, k)
    c.append(0, table[:, :0], ints(cuda_dev, 0, 0, 0), cu, k, k)
    assert int(c.status.item()) == 0 and torch.equal(c.kv, kv) and torch.equal(c.scale, scale)
    # rows that are not there are still found out
    c.attend(0, table, lens, ints(cuda_dev, 0, 0, 2, 2), q, k, k, max_len=2000, split_tokens=split)
    assert int(c.status.item()) == gs.DEV_ROWS_BAD
    c.status.zero_()
    c.append(0, table, lens, ints(cuda_dev, 0, 0, 2, 2), k, k)
    assert int(c.status.item()) == gs.DEV_ROWS_BAD and torch.equal(c.kv, kv)


@pytest.mark.parametrize("h_q,h_kv,rows", [(8, 2, 1), (4, 1, 3), (1, 1, 2), (4, 1, 1)])
def test_strides_of_single_rows_and_heads_say_nothing(cuda_dev, h_q, h_kv, rows):
    """One row, or one head: whatever stride its dimension has, as transposes and expansions leave it."""
    d = 128
    cache = ku.Cache([70], h_q, h_kv, d, 32, room=[90], seed=rows)
    c = ku.gpu_cache(cache, cuda_dev)
    table, lens, cu = torch.from_numpy(cache.table).to(cuda_dev), ints(cuda_dev, 70), ints(cuda_dev, 0, rows)
    g = torch.Generator(device=cuda_dev).manual_seed(rows)
    plain = [torch.randn((rows, h, d), generator=g, device=cuda_dev).to(torch.bfloat16) for h in (h_q, h_kv, h_kv)]

    def odd(x):
        stride = [x.stride(0) if rows > 1 else 8, d if x.shape[1] > 1 else 1, 1]
        y = torch.empty_strided(x.shape, stride, dtype=x.dtype, device=x.device)
        return y.copy_(x)

    strange = [odd(x) for x in plain]
    assert any(x.stride() != y.stride() for x, y in zip(plain, strange))
    want = c.attend(0, table, lens, cu, *plain, max_len=70, max_rows=rows, want_lse=True)
    got = c.attend(0, table, lens, cu, *strange, max_len=70, max_rows=rows, want_lse=True, out=odd(plain[0]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    before = c.kv.clone(), c.scale.clone()
    c.append(0, table, lens, cu, plain[1], plain[2])
    after = c.kv.clone(), c.scale.clone()
    c.kv.copy_(before[0])
    c.scale.copy_(before[1])
    c.append(0, table, lens, cu, strange[1], strange[2])
    assert int(c.status.item()) == 0 and torch.equal(c.kv, after[0]) and torch.equal(c.scale, after[1])
    assert not torch.equal(c.kv, before[0])


def test_entry_points_by_their_own_names(cuda_dev):
    """The binding's kv8_attend, kv8_append and kv8_copy_pages do what the handle's calls do, on any stream, and
    raise on the status codes."""
    from speculative_decoding_hybrid_gb300 import binding as gs
    cache = ku.Cache([300, 40], 8, 2, 128, 32, room=[310, 50], seed=7)
    c, e = ku.gpu_cache(cache, cuda_dev), ku.gpu_cache(cache, cuda_dev)
    table, lens = torch.from_numpy(cache.table).to(cuda_dev), ints(cuda_dev, 300, 40)
    cu, acc = ints(cuda_dev, 0, 4, 7), ints(cuda_dev, 2, 0)
    g = torch.Generator(device=cuda_dev).manual_seed(7)
    q, k, v = (torch.randn((7, h, 128), generator=g, device=cuda_dev).to(torch.bfloat16) for h in (8, 2, 2))
    want, want_lse = c.attend(0, table, lens, cu, q, k, v, max_len=300, max_rows=4, split_tokens=128, want_lse=True)
    need = gs.kv8_attend_workspace_bytes(e.c, 2, 300, 4, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse = torch.zeros_like(q), torch.zeros((7, 8), device=cuda_dev)
        ws = torch.empty((need,), dtype=torch.uint8, device=cuda_dev)
        args = (e.c, 0, 2, 7, cu, lens, table, table.shape[1], table.stride(0), q, q.stride(0), k, k.stride(0), v,
                v.stride(0), o, o.stride(0), lse, 300, 4, 128, ws)
        gs.kv8_attend(*args, need, e.status)
        gs.kv8_append(e.c, 0, 2, 7, cu, lens, table, table.shape[1], table.stride(0), k, k.stride(0), v, v.stride(0),
                      acc, 4, e.status)
        moves = ints(cuda_dev, int(cache.table[0, 9])), ints(cuda_dev, int(cache.table[0, 0]))
        gs.kv8_copy_pages(e.c, 1, *moves, e.status, stream=side)
    side.synchronize()
    c.append(0, table, lens, cu, k, v, accept_len=acc, max_rows=4)
    c.copy_pages(*moves)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert torch.equal(c.kv, e.kv) and torch.equal(c.scale, e.scale) and int(e.status.item()) == 0
    with pytest.raises(gs.GdnError):
        gs.kv8_attend(*args, need - 16, e.status)
    with pytest.raises(gs.GdnError):
        gs.kv8_copy_pages(e.c, -1, *moves, e.status)
