"""The prompt side on the host: room for a status word, tensors that are not on a GPU (no GPU: nothing is launched)."""
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
