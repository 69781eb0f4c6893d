"""The prompt side's calls run on their rows' device, whichever is the current one, and take that device's streams only.
(One device is all there is here: what the calls take for the current one is replaced.)"""
import pytest
import torch

import kv_util as ku
import prompt_util as pu
from gpu_util import build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def calls(dev):
    from speculative_decoding_hybrid_gb300.prefill import Rope, attend_prompts
    cache = ku.Cache([1000, 300], 4, 1, 128, 32, seed=4)
    t, _ = pu.rows_of(150, 4, 1, 128, 0)
    q, k, v = pu.split(t.to(dev), 4, 1, 128)
    c = ku.gpu_cache(cache, dev)
    table, lens, cu = torch.from_numpy(cache.table).to(dev), pu.dev32(cache.lens, dev), pu.dev32([0, 50, 150], dev)
    rope = Rope(128, 64, device=dev)
    return {
        "rotate": lambda **kw: rope.rotate(q, k, cu, lens, c.status, **kw),
        "attend_prompts": lambda **kw: attend_prompts(q, k, v, cu, 150, c.status, want_lse=True, **kw),
        "attend_chunk": lambda **kw: c.attend_chunk(0, table, lens, cu, q, k, v, 1000, 150, want_lse=True, **kw),
    }


@pytest.mark.parametrize("name", ["rotate", "attend_prompts", "attend_chunk"])
@pytest.mark.parametrize("on", ["given", "current"])
def test_another_device_is_current(cuda_dev, monkeypatch, name, on):
    from speculative_decoding_hybrid_gb300 import kvcache, prefill
    call = calls(cuda_dev)[name]
    ref = call()
    index, asked = torch.cuda.current_device(), []

    def current():
        asked.append(1)
        return index + 1 if len(asked) == 1 else index
    monkeypatch.setattr(prefill, "_current_device", current)
    monkeypatch.setattr(kvcache, "_current_device", current)
    kw = {}
    if on == "given":
        kw["stream"] = torch.cuda.Stream()
        kw["stream"].wait_stream(torch.cuda.current_stream())
    got = call(**kw)
    torch.cuda.synchronize()
    assert len(asked) == 2 and all(torch.equal(x, y) for x, y in zip(ref, got))


@pytest.mark.parametrize("name", ["rotate", "attend_prompts", "attend_chunk"])
def test_a_stream_of_another_device_is_refused(cuda_dev, name):
    class Elsewhere:
        device_index, cuda_stream = torch.cuda.current_device() + 1, 0
    call = calls(cuda_dev)[name]
    before = torch.cuda.current_stream()
    with pytest.raises(ValueError, match="rows' device"):
        call(stream=Elsewhere())
    assert torch.cuda.current_stream() == before
