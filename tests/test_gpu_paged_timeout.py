"""Waits that run out in the attention over 8-bit pages: a stage of the ring of keys
never comes back (the test hook that the decode step has too), as if a warp were
lost. Every wait is bounded, so the launch ends, records TP_ERR_TIMEOUT, and the
workspace serves again once it is set up anew."""
import time

import pytest

from tests import _paged as K

pytestmark = pytest.mark.gpu

L = K.Layout
# more keys for a warp, or a CTA, than its ring has stages: (layout, page, new, cached, max_new)
CASES = {
    "one_token": (L(32, 8, 128, 4), 64, [1] * 20, [1500] * 20, 1),
    "one_token_64": (L(14, 2, 64, 2), 16, [1] * 90, [2000] * 90, 1),
    "few_tokens": (L(32, 8, 128, 1), 32, [4] * 20, [1500] * 20, 4),
    "prompts": (L(32, 8, 128, 4), 64, [64] * 8, [1500] * 8, 0),
    "prompts_64": (L(8, 8, 64, 1), 32, [140] * 12, [2000] * 12, 0),
}


@pytest.mark.parametrize("name", CASES)
def test_a_lost_stage_times_out_and_the_workspace_recovers(gpu_lib, name):
    import torch
    lay, page, new, cached, max_new = CASES[name]
    d = K.OnDevice(gpu_lib, K.Batch(lay, new, cached, page), max_new)
    first = d.attend().clone()
    assert d.status() == 0
    gpu_lib.tp_debug_withhold_arrival(d.plan, True)
    try:
        t0 = time.monotonic()
        d.attend()
        torch.cuda.synchronize()                # the launch ends: its waits are bounded
        took = time.monotonic() - t0
    finally:
        gpu_lib.tp_debug_withhold_arrival(d.plan, False)
    assert d.status() == gpu_lib.binding.TP_ERR_TIMEOUT
    assert 0.9 < took < 30.0, took
    gpu_lib.tp_paged_workspace_init(d.plan, d.ws, d.nbytes)
    d.out.fill_(7.0)
    d.attend()
    assert d.status() == 0
    assert torch.equal(d.out, first)
