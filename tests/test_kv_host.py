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
