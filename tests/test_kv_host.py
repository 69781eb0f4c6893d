"""The host side of the paged 8-bit cache without a GPU: streams of uploads, page tables of other types."""
import contextlib

import numpy as np
import pytest


@pytest.fixture(scope="module")
def gs():
    from speculative_decoding_hybrid_gb300 import build
    build.build()
    from speculative_decoding_hybrid_gb300 import binding
    return binding


def test_upload_goes_to_the_cache_devices_stream(gs, monkeypatch):
    """The current stream of the cache's own device, or the copy that `_staged` waits for is another's."""
    import torch

    from speculative_decoding_hybrid_gb300 import kvcache
    asked, used, recorded = [], [], []

    class Event:
        def record(self, *a):
            recorded.append(used[-1])

        def synchronize(self):
            pass

    def stream(s):
        used.append(s)
        return contextlib.nullcontext()

    monkeypatch.setattr(kvcache.torch.cuda, "current_stream", lambda device=None: asked.append(device) or "stream")
    monkeypatch.setattr(kvcache.torch.cuda, "stream", stream)
    monkeypatch.setattr(kvcache.torch.cuda, "Event", Event)
    p = kvcache.PagedKv(1, 8, 3, 64, 4, 2, 64, page_tokens=16, device="cpu")
    p.reserve([1], [20])
    p.advance([1], [20])
    table, length = p.upload([1, 0])
    assert asked == [torch.device("cpu")] and used == ["stream"] and recorded == ["stream"]
    assert length.tolist() == [20, 0] and table[0, :2].tolist() == p.tables[1, :2].tolist()


def test_page_tables_are_int32_rows(gs):
    """What C would read past, or as something else, is refused before it gets there; nothing changes."""
    pool = gs.Pool(8)
    good = np.full(4, -1, np.int32)
    n, _ = gs.kv8_pages_reserve(pool, good, 0, 0, 20, 16)
    before = pool.free_list(), good.copy()
    wide = np.full((2, 4), -1, np.int32)
    for bad in (np.full(4, -1, np.int64), np.full(4, -1, np.int16), np.full(8, -1, np.int32)[::2],
                np.full((2, 2), -1, np.int32), [-1] * 4):
        for call in (lambda: gs.kv8_pages_reserve(pool, bad, 0, 0, 20, 16),
                     lambda: gs.kv8_pages_fork(pool, bad, 2, 20, 16, wide[0]),
                     lambda: gs.kv8_pages_fork(pool, good, n, 20, 16, bad),
                     lambda: gs.kv8_pages_free(pool, bad, 1)):
            with pytest.raises(ValueError):
                call()
    counts = np.zeros(2, np.int32)
    for tables, used in ((wide.astype(np.int64), counts), (wide[:, ::2], counts), (wide, counts.astype(np.int64)),
                         (wide, counts[:1]), (wide[0], counts), (wide, np.zeros(4, np.int32)[::2])):
        with pytest.raises(ValueError):
            gs.kv8_pages_compact(pool, tables, used)
    assert pool.free_list() == before[0] and (good == before[1]).all() and (wide == -1).all()
    with pytest.raises(gs.GdnError):
        gs.kv8_pages_free(pool, good, 5)                  # more pages than the row has entries
    with pytest.raises(gs.GdnError):
        gs.kv8_pages_fork(pool, good, 5, 70, 16, wide[0])
