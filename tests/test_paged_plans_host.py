"""Caches in pages that were made for one plan, in the calls of another (no GPU:
the refusal precedes the call into the library)."""
import pytest

import megatron_tensor_block_gb300 as tb
from megatron_tensor_block_gb300 import binding as B
from tests import _packed as K

A, FAR = 1 << 20, 1 << 24                        # aligned addresses that nothing reads


def plan(heads, kv_heads, d, tp):
    return tb.tp_plan(K.plan_desc(tb, K.Layout(heads, kv_heads, d, tp), 4, 64, 100), tp)


def caches(p, monkeypatch):
    """A PagedKV of tensors on the CPU."""
    import torch
    B._Torch.device()
    monkeypatch.setattr(B._Torch, "device", classmethod(lambda cls: -1))
    pool = [torch.zeros(3, p.hkv_shard, 16, p.head_dim, dtype=torch.uint8) for _ in range(p.tp)]
    scale = [torch.ones(3, p.hkv_shard) for _ in range(p.tp)]
    return tb.PagedKV(p, pool, pool, scale, scale, torch.zeros(4, 2, dtype=torch.int32))


@pytest.mark.parametrize("other", [(16, 8, 64, 2), (8, 2, 64, 2), (8, 4, 128, 2), (8, 4, 64, 1), (8, 4, 64, 4)])
def test_caches_of_another_plan_are_refused(monkeypatch, other):
    kv, p = caches(plan(8, 4, 64, 2), monkeypatch), plan(*other)
    for x in (kv, kv.at(kv.pages)):
        with pytest.raises(ValueError, match="expected the plan's"):
            tb.tp_attn_paged(p, A, x, A, A, 4, 64, FAR, A, tb.tp_paged_workspace_bytes(p), stream=0)
        with pytest.raises(ValueError, match="expected the plan's"):
            tb.tp_kv_append_paged(p, None, A, A, x, A, A, 4, 64, stream=0)


def test_plans_of_the_same_heads_share_caches(monkeypatch):
    """What matters is shards, KV heads and features: the struct is passed on."""
    kv, p = caches(plan(8, 4, 64, 2), monkeypatch), plan(16, 4, 64, 2)
    assert B._paged(p, kv, 4, -1)._obj is kv.struct
