"""Workspace sizes (no GPU). The packed calls' scratch lies at the end of a
workspace: the calls that were there before them take workspaces of the sizes
that they had, which are written down here."""
import pytest

import megatron_tensor_block_gb300 as tb
import synth
from megatron_tensor_block_gb300 import binding as B
from megatron_tensor_block_gb300.runtime import desc_of
from tests import _packed as K

A = 1 << 24
L = K.Layout
# layout, max_batch, max_tokens, max_kv, bytes of the workspace without packed batches
PLANS = [
    (L(32, 8, 128, 4), 8, 8, 4096, 26194176),
    (L(32, 8, 128, 1), 4, 8192, 8192, 258019840),
    (L(32, 8, 128, 8), 64, 2048, 4096, 265816576),
    (L(14, 2, 64, 2), 4, 64, 100, 1147136),
    (L(14, 2, 64, 1), 4, 2048, 2048, 19880192),
    (L(3, 3, 64, 1), 1, 1, 1, 174848),
]
WORKLOADS = {"qwen25_05b_decode_tp2": 2526464, "llama3_8b_decode_tp4": 22695680, "llama3_8b_prefill_tp8": 1050873856}


def plans():
    for lay, b, t, kv, n in PLANS:
        yield tb.tp_plan(K.plan_desc(tb, lay, b, t, kv), lay.tp), n
    for name, n in WORKLOADS.items():
        w = synth.WORKLOADS[name]
        yield tb.tp_plan(desc_of(w), w.tp), n


def status(call):
    with pytest.raises(tb.TpError) as e:
        call()
    return e.value.status


def test_a_workspace_without_the_packed_scratch_serves_the_other_calls():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the calls must fail for want of a device")
    for p, n in plans():
        kv = ([A] * p.tp, [A] * p.tp)
        for nbytes, want in ((n, B.TP_ERR_UNSUPPORTED), (n - 1, B.TP_ERR_CAPACITY)):
            assert status(lambda: tb.tp_workspace_init(p, A, nbytes, stream=0)) == want
            for mode in (B.TP_MODE_DECODE, B.TP_MODE_PREFILL):
                assert status(lambda: tb.tp_block_forward(p, {}, kv, A, 2 * A, A, 1, 1, mode, None, A, nbytes, stream=0)) == want


def test_packed_calls_need_their_scratch():
    for p, n in plans():
        kv = ([A] * p.tp, [A] * p.tp)
        assert p.workspace_bytes > n
        for nbytes in (n, p.workspace_bytes - 1):
            assert status(lambda: tb.tp_attn_packed(p, A, kv, A, A, 1, 1, 2 * A, A, nbytes, stream=0)) == B.TP_ERR_CAPACITY
            assert status(lambda: tb.tp_block_forward_packed(p, {}, kv, A, 2 * A, A, A, 1, 1, A, nbytes,
                                                             stream=0)) == B.TP_ERR_CAPACITY


def test_large_prefill_plans_hold_partial_results_where_other_buffers_lie():
    w = synth.WORKLOADS["llama3_8b_prefill_tp8"]
    for tp, n in ((1, 578228224), (2, 645599232), (4, 780341248), (8, 1050873856)):
        p = tb.tp_plan(desc_of(w), tp)
        assert n < p.workspace_bytes < 1.01 * n


def test_a_plan_object_around_a_bare_handle():
    # as it could be made before it kept sizes: every call but the packed ones takes it
    lay, b, t, kv, n = PLANS[0]
    made = tb.tp_plan(K.plan_desc(tb, lay, b, t, kv), lay.tp)
    bare = tb.Plan(made.handle)
    try:
        assert tb.tp_plan_get_info(bare) == tb.tp_plan_get_info(made)
        assert bare.workspace_bytes == made.workspace_bytes
        assert status(lambda: tb.tp_block_forward(bare, {}, None, A, A, A, 1, 1, B.TP_MODE_DECODE, None, A, n, stream=0)) \
            == B.TP_ERR_INVALID_ARG
        caches = ([A] * lay.tp, [A] * lay.tp)
        with pytest.raises(ValueError, match="description"):
            tb.tp_attn_packed(bare, A, caches, A, A, 1, 1, 2 * A, A, n, stream=0)
        with pytest.raises(ValueError, match="description"):
            tb.tp_logits_process(bare, A, 1, 2 * A, stream=0)
    finally:
        bare.handle = None                       # `made` owns it
