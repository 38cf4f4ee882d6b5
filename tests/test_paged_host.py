"""Argument checks of the rotary embedding and the calls around 8-bit pages, and
the oracle's own e4m3 and rotations (no GPU): each refusal precedes any launch,
so the made-up addresses are never read."""
import math

import numpy as np
import pytest

import megatron_tensor_block_gb300 as tb
from megatron_tensor_block_gb300 import binding as B
from tests import _paged as K

LAY = K.Layout(14, 2, 64, 2)
A, FAR = 1 << 20, 1 << 24                        # aligned addresses that nothing reads


def plan(**kw):
    return tb.tp_plan(K.plan_desc(tb, LAY, 4, 64, 100, **kw), LAY.tp)


def rows(p=A, token=64 * 7, shard=64 * 64 * 7):
    return B.tp_rows(p, token, shard)


def struct(**kw):
    s = B.tp_paged_kv(B._P8(*[A] * 2), B._P8(*[A] * 2), B._P8(*[A] * 2), B._P8(*[A] * 2), A, 10, 16, 8)
    for name, (i, x) in kw.pop("shard", {}).items():
        getattr(s, name)[i] = x
    for name, x in kw.items():
        setattr(s, name, x)
    return s


def status(call, *args):
    st = getattr(tb.load(), call)(*args)
    return st


def ref(x):
    return None if x is None else B.C.byref(x)


GOOD = dict(rot_dim=64, layout=0, scaling=0, theta=1e4)


def rope_call(p, rope=GOOD, q="rows", k="rows", cu=A, pos=A, Bn=4, T=64, q_out=FAR, k_out=2 * FAR, word=None):
    q = rows() if q == "rows" else q
    k = rows(A + (1 << 21), 64, 64 * 64) if k == "rows" else k
    return status("tp_rope_packed", p.handle, ref(tb.tp_rope(**rope)) if rope is not None else None, ref(q), ref(k), cu, pos, Bn, T,
                  q_out, k_out, word, None)


ROPES = [
    dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=80), dict(rot_dim=-16), dict(layout=2), dict(scaling=4), dict(scaling=-1),
    dict(theta=0.5), dict(theta=float("nan")), dict(theta=float("inf")), dict(scaling=1, factor=0.5), dict(scaling=1),
    dict(scaling=1, factor=float("nan")), dict(scaling=2, factor=2, low=4, high=4, original=10),
    dict(scaling=2, factor=2, low=0, high=4, original=10), dict(scaling=2, factor=2, low=1, high=4, original=0),
    dict(scaling=3, factor=2, low=1, high=float("inf"), original=9), dict(scaling=3, factor=2, low=1, high=32, original=9, theta=1.0),
    dict(attn_factor=-1.0), dict(attn_factor=float("nan")), dict(attn_factor=1e7),
]


@pytest.mark.parametrize("kw", ROPES, ids=[str(i) for i in range(len(ROPES))])
def test_ropes_outside_their_ranges_are_refused(kw):
    assert rope_call(plan(), dict(GOOD, **kw)) == B.TP_ERR_INVALID_ARG


ROPE_REFUSALS = [
    (dict(rope=None), B.TP_ERR_NULL), (dict(q=None, k=None, q_out=None, k_out=None), B.TP_ERR_NULL), (dict(q_out=None), B.TP_ERR_NULL),
    (dict(k=None), B.TP_ERR_NULL), (dict(cu=None), B.TP_ERR_NULL), (dict(pos=None), B.TP_ERR_NULL), (dict(Bn=5), B.TP_ERR_SHAPE),
    (dict(Bn=0), B.TP_ERR_SHAPE), (dict(T=65), B.TP_ERR_SHAPE), (dict(T=0), B.TP_ERR_SHAPE), (dict(cu=A + 2), B.TP_ERR_ALIGN),
    (dict(q_out=FAR + 8), B.TP_ERR_ALIGN), (dict(word=A + 1), B.TP_ERR_ALIGN), (dict(q=rows(0)), B.TP_ERR_NULL),
    (dict(q=rows(A + 8)), B.TP_ERR_ALIGN), (dict(q=rows(token=64 * 7 + 4)), B.TP_ERR_ALIGN),
    (dict(q=rows(shard=64 * 64 * 7 + 4)), B.TP_ERR_ALIGN), (dict(q=rows(token=64 * 7 - 8)), B.TP_ERR_SHAPE),
    (dict(q=rows(shard=64)), B.TP_ERR_SHAPE), (dict(q=rows(token=2 ** 62)), B.TP_ERR_SHAPE),
    (dict(q_out=A + 1024), B.TP_ERR_INVALID_ARG), (dict(q=rows(token=64 * 7 + 8), q_out=A), B.TP_ERR_INVALID_ARG),
    (dict(k_out=FAR), B.TP_ERR_INVALID_ARG), (dict(k_out=A), B.TP_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,want", ROPE_REFUSALS, ids=[str(i) for i in range(len(ROPE_REFUSALS))])
def test_rope_refuses(kw, want):
    assert rope_call(plan(), **kw) == want


def append_call(p, rope=GOOD, q=None, k="rows", v="rows", kv="kv", cu=A, pos=A, Bn=4, T=64, q_out=None, word=None):
    k, v = (rows(A + (1 << 21), 64, 64 * 64) if x == "rows" else x for x in (k, v))
    return status("tp_kv_append_paged", p.handle, ref(tb.tp_rope(**rope)) if rope is not None else None, ref(q), ref(k), ref(v),
                  ref(struct() if kv == "kv" else kv), cu, pos, Bn, T, q_out, word, None)


PAGES = [
    (dict(page=8), B.TP_ERR_INVALID_ARG), (dict(page=48), B.TP_ERR_INVALID_ARG), (dict(page=256), B.TP_ERR_INVALID_ARG),
    (dict(n_pages=0), B.TP_ERR_SHAPE), (dict(n_pages=2 ** 27), B.TP_ERR_SHAPE), (dict(width=0), B.TP_ERR_SHAPE),
    (dict(width=2 ** 27), B.TP_ERR_SHAPE), (dict(pages=None), B.TP_ERR_NULL), (dict(pages=A + 2), B.TP_ERR_ALIGN),
    (dict(shard=dict(k=(1, 0))), B.TP_ERR_NULL), (dict(shard=dict(v_scale=(0, 0))), B.TP_ERR_NULL),
    (dict(shard=dict(v=(1, A + 8))), B.TP_ERR_ALIGN), (dict(shard=dict(k_scale=(0, A + 2))), B.TP_ERR_ALIGN),
]


def attend_call(p, q=A, kv="kv", cu=A, pos=A, Bn=4, T=64, max_new=0, out=FAR, ws=A, nbytes=None):
    nbytes = tb.tp_paged_workspace_bytes(p) if nbytes is None else nbytes
    return status("tp_attn_paged", p.handle, q, ref(struct() if kv == "kv" else kv), cu, pos, Bn, T, max_new, out, ws, nbytes, None)


@pytest.mark.parametrize("kw,want", PAGES, ids=[str(i) for i in range(len(PAGES))])
def test_pages_outside_their_ranges_are_refused(kw, want):
    assert append_call(plan(), kv=struct(**kw)) == want
    assert attend_call(plan(), kv=struct(**kw)) == want


APPEND_REFUSALS = [
    (dict(k=None), B.TP_ERR_NULL), (dict(v=None), B.TP_ERR_NULL), (dict(kv=None), B.TP_ERR_NULL), (dict(cu=None), B.TP_ERR_NULL),
    (dict(q=rows()), B.TP_ERR_NULL), (dict(q_out=FAR), B.TP_ERR_NULL), (dict(q=rows(), q_out=FAR, rope=None), B.TP_ERR_INVALID_ARG),
    (dict(q=rows(), q_out=A + 64), B.TP_ERR_INVALID_ARG), (dict(q=rows(), q_out=A + (1 << 21)), B.TP_ERR_INVALID_ARG),
    (dict(v=rows(A + 8, 64, 64 * 64)), B.TP_ERR_ALIGN), (dict(k=rows(A, 60, 64 * 64)), B.TP_ERR_SHAPE), (dict(Bn=5), B.TP_ERR_SHAPE),
    (dict(T=65), B.TP_ERR_SHAPE), (dict(rope=dict(GOOD, layout=7)), B.TP_ERR_INVALID_ARG), (dict(word=A + 2), B.TP_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,want", APPEND_REFUSALS, ids=[str(i) for i in range(len(APPEND_REFUSALS))])
def test_append_refuses(kw, want):
    assert append_call(plan(), **kw) == want


ATTEND_REFUSALS = [
    (dict(q=None), B.TP_ERR_NULL), (dict(out=None), B.TP_ERR_NULL), (dict(ws=None), B.TP_ERR_NULL), (dict(kv=None), B.TP_ERR_NULL),
    (dict(pos=None), B.TP_ERR_NULL), (dict(Bn=0), B.TP_ERR_SHAPE), (dict(T=65), B.TP_ERR_SHAPE), (dict(max_new=-1), B.TP_ERR_SHAPE),
    (dict(nbytes=100), B.TP_ERR_CAPACITY), (dict(q=A + 8), B.TP_ERR_ALIGN), (dict(out=FAR + 2), B.TP_ERR_ALIGN),
    (dict(ws=A + 4), B.TP_ERR_ALIGN), (dict(out=A), B.TP_ERR_INVALID_ARG), (dict(out=A + 64 * 14 * 64 * 2 - 16), B.TP_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,want", ATTEND_REFUSALS, ids=[str(i) for i in range(len(ATTEND_REFUSALS))])
def test_attention_refuses(kw, want):
    assert attend_call(plan(), **kw) == want


def test_only_bf16_plans_have_pages():
    p = plan(dtype=tb.TP_F32)
    assert append_call(p) == B.TP_ERR_UNSUPPORTED
    assert attend_call(p, nbytes=1 << 30) == B.TP_ERR_UNSUPPORTED
    with pytest.raises(tb.TpError) as e:
        tb.tp_paged_workspace_bytes(p)
    assert e.value.status == B.TP_ERR_UNSUPPORTED


def test_workspace_refuses():
    p = plan()
    n = tb.tp_paged_workspace_bytes(p)
    for ws, nbytes, want in ((None, n, B.TP_ERR_NULL), (A, n - 1, B.TP_ERR_CAPACITY), (A + 8, n, B.TP_ERR_ALIGN)):
        assert status("tp_paged_workspace_init", p.handle, ws, nbytes, None) == want
    assert status("tp_paged_workspace_bytes", p.handle, None) == B.TP_ERR_NULL


def test_binding_refuses_tensors_that_do_not_fit():
    import torch
    p = plan()
    k = torch.zeros(2, 64, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        tb.tp_rope_packed(p, tb.tp_rope(), A, A, 4, 64, k=k.float(), k_out=FAR, stream=0)
    with pytest.raises(ValueError, match="expected"):
        tb.tp_rope_packed(p, tb.tp_rope(), A, A, 4, 64, k=k[:, :63], k_out=FAR, stream=0)
    pool = [torch.zeros(3, 1, 16, 64, dtype=torch.uint8)] * 2
    scale, table = [torch.ones(3, 1)] * 2, torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        tb.PagedKV(p, pool[:1], pool, scale, scale, table)
    with pytest.raises(TypeError):
        tb.PagedKV(p, [x.float() for x in pool], pool, scale, scale, table)
    with pytest.raises(ValueError):
        tb.PagedKV(p, pool, pool, scale, [x[:2] for x in scale], table)


def test_e4m3_of_the_oracle():
    import torch
    x = np.concatenate([np.random.default_rng(0).standard_normal(20000) * 10.0 ** np.linspace(-4, 2, 20000), K.DECODE[:127],
                        (K.DECODE[:126] + K.DECODE[1:127]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (K.encode(x) == want).all()
    assert (K.encode([np.inf, np.nan, -np.inf]) & 127 == 127).all()


def test_scales_of_the_oracle():
    for x, e in ((448.0, 0), (448.0 + 2 ** -40, 1), (1.75, -8), (3.5, -7), (1.0, -8), (0.0, -60), (2.0 ** -70, -60), (3e38, 120)):
        assert K.exponent(np.array([x]), 1.0)[0] == e


def test_rotations_of_the_oracle():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, 3, 2, 64))
    for layout in (0, 1):
        r = K.rope_args(rot=32, layout=layout, theta=1e4)
        y, _ = K.rotate(x, [0, 5, 9], r, 1.0)
        assert (y[:, 0] == x[:, 0]).all() and (y[..., 32:] == x[..., 32:]).all()
        a, b = (0, 16) if layout == 0 else (0, 1)
        z = (x[0, 1, 0, a] + 1j * x[0, 1, 0, b]) * np.exp(5j)
        assert abs(y[0, 1, 0, a] - z.real) < 1e-12 and abs(y[0, 1, 0, b] - z.imag) < 1e-12
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    f, m = K.frequencies(K.rope_args(scaling=2, factor=8, low=1, high=4, original=8192, theta=5e5), 128, 1.0)
    g, _ = K.frequencies(K.rope_args(theta=5e5), 128, 1.0)
    wave = 2 * math.pi / g
    assert np.allclose(f[wave < 2048], g[wave < 2048]) and np.allclose(f[wave > 8192], g[wave > 8192] / 8) and m == 1
    f, m = K.frequencies(K.rope_args(scaling=3, factor=4, low=1, high=32, original=32768, theta=1e6), 64, 1.0)
    g, _ = K.frequencies(K.rope_args(theta=1e6), 64, 1.0)
    assert f[0] == g[0] and abs(f[-1] - g[-1] / 4) < 1e-18 and abs(m - 1.1386294361) < 1e-9
