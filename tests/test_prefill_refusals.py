"""The prompt side on the host: room for a status word, tensors that are not on a GPU, frequencies scaled by parts (no GPU:
nothing is launched)."""
import math

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def gs():
    from speculative_decoding_hybrid_gb300 import build
    build.build()
    from speculative_decoding_hybrid_gb300 import binding
    return binding


def test_cut_work_has_room_for_a_status_word(gs):
    """Behind its units' sums, statistics and records: without dev_status the join has no other word to go by."""
    for h_q, d, n in ((4, 64, 2000), (4, 128, 3000), (2, 256, 1500)):
        need = gs.attn_prompts_workspace_bytes(gs.attn_dims(h_q, 1, d, 0, 0.1), 1, n, n)
        stages = 1 if d == 256 else 2
        per = stages * (128 // h_q)
        units = min(-(-n // per), n // per + 1)
        assert need > 0 and (need - units * 32) % (units * stages * 128 * (d * 4 + 8)) == 16


def calls(gs, device):
    """Each call with all of its tensors on `device`."""
    from speculative_decoding_hybrid_gb300.kvcache import PagedKv
    from speculative_decoding_hybrid_gb300.prefill import Rope, attend_prompts
    x = lambda h: torch.zeros((8, h, 64), dtype=torch.bfloat16, device=device)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device=device)
    cu, status = i(0, 8), i(0)
    yield "rotate", lambda **kw: Rope(64, device=device).rotate(x(4), x(2), cu, None, status, **kw)
    yield "rotate in place", lambda **kw: Rope(64, device=device).rotate(x(4), None, cu, i(5), status, in_place=True, **kw)
    yield "attend_prompts", lambda **kw: attend_prompts(x(4), x(2), x(2), cu, 8, status, **kw)
    cache = PagedKv(1, 4, 1, 64, 4, 2, 64, page_tokens=16, device=device)
    yield "attend_chunk", lambda **kw: cache.attend_chunk(0, i(0, 1).view(1, 2), i(10), cu, x(4), x(2), x(2), 10, 8, **kw)


def test_tensors_that_are_all_on_the_cpu_are_refused(gs, monkeypatch):
    """All of one device, which is none that the library launches on; whatever the current device is."""
    from speculative_decoding_hybrid_gb300 import kvcache, prefill
    for module in (kvcache, prefill):
        monkeypatch.setattr(module, "_current_device", lambda: 0)
    for name, call in calls(gs, "cpu"):
        for kw in (dict(), dict(stream=0)):
            with pytest.raises(ValueError, match="on a GPU"):
                call(**kw)


def test_the_line_of_scaling_by_parts(gs):
    """Between its ends a frequency's share goes by how often it turns in the trained length: at a quarter of the way
    from `slow` to `fast` a quarter of it stays and three quarters are divided by the factor."""
    from speculative_decoding_hybrid_gb300.prefill import Rope, rope_frequencies
    for slow, fast, factor in ((1.0, 32.0, 8.0), (1.0, 4.0, 16.0), (2.5, 20.0, 3.0)):
        for share in (0.0, 0.25, 0.5, 0.9, 1.0):
            f = 1000.0 ** -0.5                                 # the second of two frequencies, of base 1000
            turns = slow + share * (fast - slow)
            trained = 2 * math.pi * turns / f
            kw = dict(base=1000.0, scaling="parts", factor=factor, trained=trained, slow=slow, fast=fast)
            g, m = rope_frequencies(4, **kw)
            assert abs(g[1] - (share * f + (1 - share) * f / factor)) < 1e-12 * f
            assert abs(m - (1 + 0.1 * math.log(factor))) < 1e-15
            rope = Rope(8, 4, device="cpu", **kw)
            assert np.array_equal(rope.frequencies, g) and rope.magnitude == m
    with pytest.raises(ValueError):
        Rope(8, 4, device="cpu", scaling="parts", factor=2.0, trained=100, slow=4.0, fast=4.0)
