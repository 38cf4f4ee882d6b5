"""Packed attention in caches of more than 2^31 elements with enough new tokens
for both kernels, and replays of a captured call of few rows against float64."""
import numpy as np
import pytest

from tests import _packed as K

pytestmark = pytest.mark.gpu

L = K.Layout
QWEN = L(14, 2, 64, 2)


@pytest.mark.parametrize("new,cached", [([3], [297]), ([70], [230]), ([200], [0]), ([40], [600])],
                         ids=["few_rows", "two_tiles", "a_prompt", "parts"])
def test_the_last_sequence_of_a_far_cache(gpu_lib, new, cached):
    # the sequence's rows lie behind 2^31 elements of its shard's cache; of a value that overflowed there the rows that
    # see it must get it: the wide kernel reads such values by their own addresses
    import torch
    tb = gpu_lib
    lay, rows, B = L(8, 4, 128, 1), 140000, 32
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB of device memory")
    assert (B - 1) * lay.hkv * rows * lay.d > 2 ** 31
    k = torch.zeros(B, lay.hkv, rows, lay.d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = K.Batch(lay, [0] * (B - 1) + new, [0] * (B - 1) + cached, seed=8, stale=0.0)
    end = new[0] + cached[0]
    for dst, src in ((k, small.k[0]), (v, small.v[0])):
        dst[B - 1, :, :end].copy_(torch.from_numpy(src[B - 1].astype(np.float32)))
        dst[B - 1, :, end:end + 300] = float("nan")      # what an earlier sequence left
    v[B - 1, 3, end - 2, 5] = float("inf")               # seen by the last two tokens of the last heads
    d = K.OnDevice(tb, small)
    plan = tb.tp_plan(K.plan_desc(tb, lay, B, small.T, rows), 1)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    tb.tp_workspace_init(plan, ws, plan.workspace_bytes)
    tb.tp_attn_packed(plan, d.q, ([k], [v]), d.cu, d.pos, B, small.T, d.out, ws, plan.workspace_bytes)
    assert tb.tp_get_device_status(ws) == 0
    got = d.got()
    o, bound = small.reference()
    seen = np.zeros(o.shape, bool)
    seen[0, -2:, 3 * lay.group:4 * lay.group, 5] = True
    assert (got[seen] == np.inf).all()
    assert (np.abs(got - o)[~seen] <= bound[~seen]).all()


@pytest.mark.parametrize("prefix", [0, 150])
def test_replays_of_a_call_of_few_rows_match_float64(gpu_lib, prefix):
    import torch
    tb = gpu_lib
    full = K.Batch(QWEN, [2, 1, 1], [900, 900, 900], prefix=prefix, seed=7)
    d = K.OnDevice(tb, full)
    d.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.run()
    for new, cached in (([1, 0, 1], [5, 0, 640]), ([0, 0, 4], [1, 1, 127]), ([1, 1, 1], [127, 128, 255]), ([4, 0, 0], [0, 3, 3]),
                        ([0, 0, 0], [1, 2, 3]), ([2, 1, 1], [900, 900, 900])):
        b = K.Batch(QWEN, new, cached, prefix=prefix, seed=7, max_kv=full.max_kv, stale=0.0)
        b.T, b.q, b.pk, b.pv, b.k, b.v = full.T, full.q, full.pk, full.pv, full.k, full.v
        d.cu.copy_(torch.from_numpy(b.cu))
        d.pos.copy_(torch.tensor(cached, dtype=torch.int32))
        d.out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert d.status() == 0
        K.check(d.got(), b)


@pytest.mark.parametrize("new", [[1, 2, 1], [1] * 40, [150, 90]], ids=["few_rows", "shared", "prompts"])
def test_a_prefix_of_many_rows_of_which_few_are_used(gpu_lib, new):
    # the last KV heads' rows lie behind 2^31 elements
    import torch
    tb = gpu_lib
    lay, rows = L(8, 4, 128, 1), 6_000_000
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB of device memory")
    assert (lay.hkv - 1) * rows * lay.d > 2 ** 31
    b = K.Batch(lay, new, [7 * i for i in range(len(new))], prefix=333, seed=9)
    d = K.OnDevice(tb, b)
    pk, pv = (torch.full((lay.hkv, rows, lay.d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pk[:, :333], pv[:, :333] = d.pk[0], d.pv[0]
    tb.tp_attn_prefix(d.plan, d.q, ([pk], [pv]), 333, rows, (d.k, d.v), d.cu, d.pos, b.B, b.T, d.out, d.ws, d.nbytes)
    assert d.status() == 0
    K.check(d.got(), b)
