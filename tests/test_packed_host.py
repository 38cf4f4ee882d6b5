"""Argument checks of the packed calls and the logit controls (no GPU): each
refusal precedes any launch, so the made-up addresses are never read."""
import numpy as np
import pytest

import megatron_tensor_block_gb300 as tb
from megatron_tensor_block_gb300 import binding as B
from tests import _packed as K

LAY = K.Layout(14, 2, 64, 2)
A = 1 << 20                                      # an aligned address that nothing reads


def plan(**kw):
    return tb.tp_plan(K.plan_desc(tb, LAY, 4, 64, 100, **kw), LAY.tp)


def packed(p, q=A, kv=([A, A], [A, A]), cu=A, pos=A, Bn=4, T=64, out=A + (1 << 20), ws=A, nbytes=None, prefix=None,
           prefix_len=0, prefix_rows=0):
    nbytes = p.workspace_bytes if nbytes is None else nbytes
    if prefix is None and not prefix_len:
        tb.tp_attn_packed(p, q, kv, cu, pos, Bn, T, out, ws, nbytes, stream=0)
    else:
        tb.tp_attn_prefix(p, q, prefix, prefix_len, prefix_rows, kv, cu, pos, Bn, T, out, ws, nbytes, stream=0)


REFUSALS = [
    (dict(q=None), B.TP_ERR_NULL), (dict(out=None), B.TP_ERR_NULL), (dict(cu=None), B.TP_ERR_NULL),
    (dict(pos=None), B.TP_ERR_NULL), (dict(ws=None), B.TP_ERR_NULL), (dict(kv=([A, 0], [A, A])), B.TP_ERR_NULL),
    (dict(Bn=0), B.TP_ERR_SHAPE), (dict(Bn=5), B.TP_ERR_SHAPE), (dict(T=0), B.TP_ERR_SHAPE),
    (dict(T=65), B.TP_ERR_SHAPE), (dict(nbytes=1000), B.TP_ERR_CAPACITY),
    (dict(q=A + 8), B.TP_ERR_ALIGN), (dict(out=A + (1 << 20) + 2), B.TP_ERR_ALIGN), (dict(cu=A + 2), B.TP_ERR_ALIGN),
    (dict(ws=A + 4), B.TP_ERR_ALIGN), (dict(kv=([A, A], [A, A + 8])), B.TP_ERR_ALIGN),
    (dict(out=A), B.TP_ERR_INVALID_ARG), (dict(out=A + 64 * 14 * 64 * 2 - 16), B.TP_ERR_INVALID_ARG),
    (dict(prefix=([A, A], [A, A]), prefix_len=9, prefix_rows=8), B.TP_ERR_CAPACITY),
    (dict(prefix=([A, A], [A, A]), prefix_len=-1, prefix_rows=8), B.TP_ERR_SHAPE),
    (dict(prefix=([A, A], [A, A]), prefix_len=2 ** 31 - 50, prefix_rows=2 ** 31), B.TP_ERR_SHAPE),
    (dict(prefix=([A, A], [A, A]), prefix_len=2 ** 63 - 1, prefix_rows=2 ** 63 - 1), B.TP_ERR_SHAPE),
    (dict(prefix=([A, A], [0, A]), prefix_len=8, prefix_rows=8), B.TP_ERR_NULL),
]


@pytest.mark.parametrize("kw,status", REFUSALS, ids=[str(i) for i in range(len(REFUSALS))])
def test_packed_attention_refuses(kw, status):
    with pytest.raises(tb.TpError) as e:
        packed(plan(), **kw)
    assert e.value.status == status, str(e.value)


def test_packed_calls_need_a_bf16_attention_plan():
    with pytest.raises(tb.TpError) as e:
        packed(plan(dtype=tb.TP_F32))
    assert e.value.status == B.TP_ERR_UNSUPPORTED
    moe = tb.tp_plan(dict(K.plan_desc(tb, LAY, 4, 64, 100), n_heads=0, n_kv_heads=0, head_dim=0, ffn=0, max_kv=0,
                          n_experts=4, top_k=2, expert_ffn=256, hidden=256), 2)
    with pytest.raises(tb.TpError) as e:
        B._check(tb.load().tp_attn_packed(moe.handle, A, B.C.byref(B._kv_set([A, A], [A, A])), A, A, 1, 1, 2 * A, A,
                                          moe.workspace_bytes, None))
    assert e.value.status == B.TP_ERR_INVALID_ARG


def test_prefix_pointer_is_needed_when_it_has_rows():
    p = plan()
    with pytest.raises(tb.TpError) as e:
        B._check(tb.load().tp_attn_prefix(p.handle, A, None, 8, 8, B.C.byref(B._kv_set([A, A], [A, A])), A, A, 1, 1, 2 * A, A,
                                          p.workspace_bytes, None))
    assert e.value.status == B.TP_ERR_NULL


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), B.TP_ERR_NULL), (dict(y=A), B.TP_ERR_INVALID_ARG), (dict(y=A + (1 << 20) + 4), B.TP_ERR_ALIGN),
    (dict(T=65), B.TP_ERR_SHAPE), (dict(Bn=0), B.TP_ERR_SHAPE), (dict(nbytes=100), B.TP_ERR_CAPACITY)])
def test_packed_block_refuses(kw, status):
    p = plan()
    a = dict(x=A, y=A + (1 << 20), T=64, Bn=4, nbytes=p.workspace_bytes)
    a.update(kw)
    with pytest.raises(tb.TpError) as e:
        tb.tp_block_forward_packed(p, {}, ([A, A], [A, A]), a["x"], a["y"], A, A, a["Bn"], a["T"], A, a["nbytes"], stream=0)
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("apart", [16, 64 * K.plan_desc(tb, LAY, 4, 64, 100)["hidden"] * 4 - 16])
def test_packed_block_refuses_an_output_over_its_input(apart):
    p = plan()
    for x, y in ((A, A + apart), (A + apart, A)):
        with pytest.raises(tb.TpError) as e:
            tb.tp_block_forward_packed(p, {}, ([A, A], [A, A]), x, y, A, A, 4, 64, A, p.workspace_bytes, stream=0)
        assert e.value.status == B.TP_ERR_INVALID_ARG


LOGITS = [
    (dict(logits=None), B.TP_ERR_NULL), (dict(out=None), B.TP_ERR_NULL), (dict(T=0), B.TP_ERR_SHAPE),
    (dict(tokens=A), B.TP_ERR_NULL), (dict(cu_tokens=A), B.TP_ERR_NULL), (dict(repetition=A), B.TP_ERR_NULL),
    (dict(n_prompt=A), B.TP_ERR_NULL), (dict(bias_ids=A, cu_bias=A), B.TP_ERR_NULL),
    (dict(bias_ids=A, bias_values=A), B.TP_ERR_NULL), (dict(mask_row=A), B.TP_ERR_NULL),
    (dict(mask=A, mask_rows=1), B.TP_ERR_SHAPE), (dict(mask=A, mask_row=A, mask_rows=-1), B.TP_ERR_SHAPE),
    (dict(out=A + 4), B.TP_ERR_INVALID_ARG), (dict(out=A + 2), B.TP_ERR_ALIGN), (dict(tokens=A + 1, cu_tokens=A), B.TP_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,status", LOGITS, ids=[str(i) for i in range(len(LOGITS))])
def test_logit_controls_refuse(kw, status):
    a = dict(logits=A, T=2, out=A + (1 << 20))
    a.update(kw)
    with pytest.raises(tb.TpError) as e:
        tb.tp_logits_process(plan(org_vocab=1000), stream=0, **a)
    assert e.value.status == status, str(e.value)


def test_logit_controls_need_a_head():
    with pytest.raises(tb.TpError) as e:
        tb.tp_logits_process(plan(), A, 1, 2 * A, stream=0)
    assert e.value.status == B.TP_ERR_INVALID_ARG


def test_bindings_refuse_wrong_tensors():
    import torch
    p = plan(org_vocab=1000)
    x = torch.zeros(2, 1000)
    for bad, error in ((x.double(), TypeError), (torch.zeros(1000, 2).t(), ValueError), (x[:1], ValueError), (x, ValueError)):
        with pytest.raises(error):
            tb.tp_logits_process(p, bad, 2, A, stream=0)       # wrong type, strides, size; not on a device
    with pytest.raises(ValueError):
        packed(p, kv=([A], [A]))                               # one shard's caches of two
    with pytest.raises(TypeError):
        packed(p, q=torch.zeros(2, 64, 7, 64))


def test_the_float64_attention_of_the_tests():
    # against a direct evaluation, row by row
    b = K.Batch(K.Layout(4, 2, 64, 2), [3, 0, 2], [1, 5, 0], prefix=2, seed=1)
    o, bound = b.reference()
    for t, (s, p) in enumerate([(0, 1), (0, 2), (0, 3), (2, 0), (2, 1)]):
        for r in range(2):
            for h in range(2):
                k = np.concatenate([b.pk[r, 0], b.k[r, s, 0, :p + 1]])
                v = np.concatenate([b.pv[r, 0], b.v[r, s, 0, :p + 1]])
                w = np.exp(k @ b.q[r, t, h] / 8.0)
                assert np.allclose(o[r, t, h], (w / w.sum()) @ v, rtol=1e-12, atol=1e-13)
    assert (bound > 0).all() and (bound < 0.2).all()
