"""Rotary embeddings of packed batches, appending to 8-bit pages and attention
over them against float64, element by element within the bounds that
``tests/_paged.py`` derives."""
import numpy as np
import pytest

from tests import _paged as K

pytestmark = pytest.mark.gpu

L = K.Layout
LLAMA, QWEN = L(32, 8, 128, 4), L(14, 2, 64, 2)
R = K.rope_args
WAVES = R(scaling=2, factor=8.0, low=1.0, high=4.0, original=8192, theta=5e5)
RAMP = R(scaling=3, factor=4.0, low=1.0, high=32.0, original=32768, theta=1e6)

ROPES = {
    "half": (QWEN, R(theta=1e6), [1, 5, 0, 40], [0, 9, 3, 511]),
    "half_128": (LLAMA, R(), [17, 1, 1, 30], [0, 100000, 16, 7]),
    "interleaved": (QWEN, R(layout=1, theta=1e4), [3, 1], [2, 70]),
    "part": (LLAMA, R(rot=32), [9, 2], [0, 1000]),
    "part_interleaved": (L(8, 2, 128, 2), R(rot=48, layout=1), [9, 2], [5, 1000]),
    "smallest_part": (L(3, 3, 64, 1), R(rot=16), [9, 2], [5, 1000]),
    "linear": (QWEN, R(scaling=1, factor=2.5), [20], [4000]),
    "waves": (LLAMA, WAVES, [20, 1], [0, 130000]),
    "ramp": (L(8, 2, 128, 2), RAMP, [20, 1], [0, 130000]),
    "factor": (QWEN, R(attn_factor=0.5), [20], [3]),
    "far": (L(2, 2, 64, 1), R(theta=1e4), [3, 2], [2 ** 31 - 3, 2 ** 30 + 1]),
    "before_the_first": (L(2, 2, 64, 1), R(theta=1e4), [5], [-3]),
    "many_rows": (L(8, 1, 64, 1), R(), [1300, 1, 700], [0, 5, 30]),
    "single_theta": (L(2, 2, 64, 1), R(theta=1.0), [5], [10]),
}


def rope_batch(name, seed=0):
    lay, rope, new, cached = ROPES[name]
    b = K.Batch(lay, new, [0] * len(new), extra_rows=3, seed=seed)
    b.cached = cached
    return b, rope


@pytest.mark.parametrize("name", ROPES)
def test_rope(gpu_lib, name):
    import torch
    b, rope = rope_batch(name)
    d = K.OnDevice(gpu_lib, b)
    q_out, k_out = torch.full_like(d.q, 7.0), torch.full_like(d.new_k, 7.0)
    gpu_lib.tp_rope_packed(d.plan, gpu_lib.tp_rope(**rope), d.cu, d.pos, b.B, b.T, q=d.q, q_out=q_out, k=d.new_k, k_out=k_out,
                           device_status=d.word)
    for x, got in ((b.q, q_out), (b.new_k, k_out)):
        got = got.double().cpu().numpy()
        want, err = K.rotate(x[:, :b.used], b.positions(), rope, 5e5)
        assert (np.abs(got[:, :b.used] - want) <= 2.0 ** -8 * np.abs(want) + 1.01 * err).all()
        assert (got[:, b.used:] == 7.0).all()
    assert d.word.item() == 0


@pytest.mark.parametrize("name", ["half", "part_interleaved", "far", "ramp"])
def test_rope_float32(gpu_lib, name):
    import torch
    b, rope = rope_batch(name)
    plan = gpu_lib.tp_plan(K.plan_desc(gpu_lib, b.lay, b.B, b.T, 64, dtype=gpu_lib.TP_F32), b.lay.tp)
    q = torch.from_numpy(b.q.astype(np.float32)).cuda()
    cu, pos = torch.from_numpy(b.cu).cuda(), torch.tensor(b.cached, dtype=torch.int32).cuda()
    out = torch.full_like(q, 7.0)
    gpu_lib.tp_rope_packed(plan, gpu_lib.tp_rope(**rope), cu, pos, b.B, b.T, q=q, q_out=out)
    want, err = K.rotate(b.q[:, :b.used], b.positions(), rope, 5e5)
    got = out.double().cpu().numpy()
    assert (np.abs(got[:, :b.used] - want) <= 2.0 ** -24 * np.abs(want) + 1.01 * err).all()
    assert (got[:, b.used:] == 7.0).all()


@pytest.mark.parametrize("name", ["half", "part_interleaved"])
def test_rope_in_place_and_of_pieces_of_a_fused_row(gpu_lib, name):
    import torch
    b, rope = rope_batch(name)
    d, lay = K.OnDevice(gpu_lib, b), b.lay
    rope = gpu_lib.tp_rope(**rope)
    q_out, k_out = torch.empty_like(d.q), torch.empty_like(d.new_k)
    q_out[:, b.used:], k_out[:, b.used:] = d.q[:, b.used:], d.new_k[:, b.used:]
    gpu_lib.tp_rope_packed(d.plan, rope, d.cu, d.pos, b.B, b.T, q=d.q, q_out=q_out, k=d.new_k, k_out=k_out)
    fused = torch.cat([d.q, d.new_k, d.new_v], 2).transpose(0, 1).contiguous().transpose(0, 1)     # [T][tp][heads][d]
    again_q, again_k = q_out.clone(), k_out.clone()
    gpu_lib.tp_rope_packed(d.plan, rope, d.cu, d.pos, b.B, b.T, q=fused[:, :, :lay.hq], q_out=again_q)
    gpu_lib.tp_rope_packed(d.plan, rope, d.cu, d.pos, b.B, b.T, k=fused[:, :, lay.hq:lay.hq + lay.hkv], k_out=again_k)
    assert torch.equal(again_q, q_out) and torch.equal(again_k, k_out)
    gpu_lib.tp_rope_packed(d.plan, rope, d.cu, d.pos, b.B, b.T, q=d.q, q_out=d.q, k=d.new_k, k_out=d.new_k)
    assert torch.equal(d.q, q_out) and torch.equal(d.new_k, k_out)


# name -> (layout, rope or None, page, new, cached, other arguments)
APPENDS = {
    "one_token": (QWEN, R(theta=1e6), 16, [1], [512], {}),
    "one_token_in_a_page": (QWEN, R(theta=1e6), 16, [1], [519], {}),
    "decode": (LLAMA, WAVES, 64, [1] * 40, [(37 * i) % 200 for i in range(40)], {}),
    "decode_rotated_already": (LLAMA, None, 32, [1] * 9, [0, 1, 31, 32, 33, 63, 64, 5, 100], {}),
    "prompts": (L(8, 2, 128, 2), WAVES, 32, [0, 70, 1, 33, 31, 32, 0, 130], [4, 0, 31, 40, 1, 32, 0, 15], dict(extra_rows=9)),
    "prompts_64": (QWEN, RAMP, 16, [100, 15, 16, 17, 1], [0, 1, 8, 15, 160], {}),
    "prompt_128": (L(4, 4, 128, 1), R(layout=1, rot=64), 128, [300, 129], [100, 0], {}),
    "prompt_64_128": (L(4, 1, 64, 1), R(layout=1), 128, [400], [127], {}),
    "long": (L(2, 2, 64, 1), R(), 16, [2000], [7], {}),
    "many_short": (L(2, 2, 64, 2), R(), 16, [1, 2, 0, 3] * 30, [(29 * i) % 40 for i in range(120)], {}),
    "values_behind_the_new": (QWEN, R(), 32, [1, 3, 9], [10, 1, 60], dict(stale=0x35, spread=12)),
    "small_pages_held": (QWEN, R(), 16, [3, 5], [10, 13], dict(spread=20)),
    "attn_factor": (QWEN, R(attn_factor=3.0), 16, [20], [5], {}),
    "far": (L(2, 2, 64, 1), R(theta=1e4), 128, [3], [2 ** 20 + 5], {}),
}


def check_pages(d, b, rope):
    for name, (codes, value, bound, scale) in b.appended(rope, 5e5).items():
        got = np.stack([x.cpu().numpy() for x in d.pool[name]])
        got_scale = np.stack([x.cpu().numpy() for x in d.scale[name]])
        assert (got_scale == scale).all(), name
        free = bound == 0
        same = np.where(np.isfinite(value), got == codes, (got & 127) == 127)
        assert same[free].all(), (name, np.argwhere(~same & free)[:5])
        assert (np.abs(K.DECODE[got[~free]] - value[~free]) <= bound[~free]).all(), name
        near = np.mean(got[~free] != codes[~free]) if (~free).any() else 0.0
        assert near < 1e-3, (name, near)               # a stored value a step off is one whose rounding is a close call


@pytest.mark.parametrize("name", APPENDS)
def test_append(gpu_lib, name):
    import torch
    lay, rope, page, new, cached, kw = APPENDS[name]
    b = K.Batch(lay, new, cached, page, **kw)
    d = K.OnDevice(gpu_lib, b)
    q_out = torch.full_like(d.q, 7.0)
    d.append(rope, **(dict(q=d.q, q_out=q_out) if rope else {}))
    assert d.word.item() == 0
    check_pages(d, b, rope)
    if rope:
        want = torch.full_like(d.q, 7.0)
        gpu_lib.tp_rope_packed(d.plan, gpu_lib.tp_rope(**rope), d.cu, d.pos, b.B, b.T, q=d.q, q_out=want)
        assert torch.equal(q_out, want)
    first = {n: [x.clone() for x in d.pool[n] + d.scale[n]] for n in "kv"}
    d.append(rope)                                      # the same again changes nothing
    assert all(torch.equal(x, y) for n in "kv" for x, y in zip(first[n], d.pool[n] + d.scale[n]))


def test_append_extremes(gpu_lib):
    b = K.Batch(L(2, 2, 64, 1), [20, 3], [5, 16], 16)
    b.new_k[0, 3, 0, 5], b.new_k[0, 4, 1, 7], b.new_k[0, 9, 1, 0] = np.nan, np.inf, -np.inf
    b.new_v[0, 2, 0, 1], b.new_v[0, 6, 1, 2], b.new_v[0, 7, 0, 3] = np.inf, np.nan, -np.inf
    b.new_v[0, 8, 0], b.new_v[0, 21, 0] = K.bf16(3e38), 0.0
    b.new_v[0, 20:23, 1], b.new_k[0, 20:23, 0] = 0.0, 0.0
    b.new_v[0, 20, 0], b.new_v[0, 22, 0] = K.bf16(1e-30), 0.0
    b.new_k[0, 20:23, 1] = K.bf16(2.9e38)
    d = K.OnDevice(gpu_lib, b)
    d.append(R(theta=1e4))
    check_pages(d, b, R(theta=1e4))


def test_append_outside_the_pages(gpu_lib):
    b = K.Batch(L(2, 2, 64, 1), [6, 5, 20, 4], [13, -2, 30, 0], 16, width=2)
    b.table[0, 1], b.table[3, 0] = b.n_pages, -7
    d = K.OnDevice(gpu_lib, b)
    d.append(R())
    assert gpu_lib.binding.STATUS_NAMES[d.word.item()] == "TP_ERR_CAPACITY"
    check_pages(d, b, R())


@pytest.mark.parametrize("cu", [[0, 5, 3], [1, 3, 6], [0, 3, 99], [0, -1, 6], [-4, 0, 6]])
def test_malformed_offsets_write_nothing(gpu_lib, cu):
    import torch
    b = K.Batch(L(2, 2, 64, 1), [3, 3], [5, 16], 16)
    d = K.OnDevice(gpu_lib, b)
    before = [x.clone() for n in "kv" for x in d.pool[n] + d.scale[n]]
    d.cu.copy_(torch.tensor(cu))
    q_out = torch.full_like(d.q, 7.0)
    rope = gpu_lib.tp_rope(theta=1e4)
    for call in (lambda: d.append(R(), q=d.q, q_out=q_out),
                 lambda: gpu_lib.tp_rope_packed(d.plan, rope, d.cu, d.pos, 2, 6, q=d.q, q_out=q_out, device_status=d.word)):
        d.word.zero_()
        call()
        assert gpu_lib.binding.STATUS_NAMES[d.word.item()] == "TP_ERR_SHAPE"
    d.attend()
    assert gpu_lib.binding.STATUS_NAMES[d.status()] == "TP_ERR_SHAPE"
    assert (q_out == 7).all() and (d.out == 7).all()
    assert all(torch.equal(x, y) for x, y in zip(before, [x for n in "kv" for x in d.pool[n] + d.scale[n]]))


# name -> (layout, page, new tokens, cached tokens, other arguments, max_new)
ATTENDS = {
    "one_token_alone": (L(8, 2, 128, 2), 16, [1], [0], {}, 1),
    "one_token_edges": (L(8, 2, 128, 2), 16, [1] * 9, [14, 15, 16, 30, 31, 32, 127, 128, 511], {}, 1),
    "one_token_edges_64": (QWEN, 64, [1] * 9, [14, 31, 63, 64, 65, 127, 128, 255, 511], {}, 1),
    "one_token_long": (QWEN, 32, [1, 1], [5000, 1], dict(extra_pages=3), 1),
    "one_token_many_parts": (L(8, 1, 128, 1), 128, [1], [20000], {}, 1),
    "decode": (LLAMA, 64, [1] * 30, [(131 * i) % 900 for i in range(30)], {}, 1),
    "decode_short_many": (L(4, 4, 64, 1), 16, [1] * 300, [(7 * i) % 40 for i in range(300)], {}, 1),
    "decode_empty_between": (QWEN, 16, [0, 1, 0, 0, 1, 1, 0], [5, 70, 0, 9, 0, 33, 100], {}, 0),
    "few_tokens": (L(8, 2, 128, 2), 16, [2, 4, 1, 3], [100, 31, 0, 256], {}, 4),
    "few_tokens_group8": (L(8, 1, 64, 1), 32, [2, 2, 1], [100, 31, 700], {}, 2),
    "few_tokens_group1": (L(2, 2, 128, 1), 16, [16, 9, 1, 8], [100, 31, 0, 256], {}, 16),
    "group3": (L(6, 2, 64, 1), 16, [5, 1, 2], [90, 31, 700], {}, 5),
    "group5": (L(5, 1, 128, 1), 64, [3, 1, 2], [90, 31, 300], {}, 3),
    "more_than_a_few": (L(8, 2, 128, 2), 16, [5, 8, 1, 17], [100, 31, 0, 256], {}, 0),
    "prompts": (L(8, 2, 128, 2), 32, [0, 31, 32, 33, 64, 65, 130], [0] * 7, {}, 0),
    "prompts_cached": (LLAMA, 16, [5, 64, 129, 1, 40], [0, 1, 127, 300, 128], dict(extra_pages=2), 129),
    "prompts_qwen": (QWEN, 64, [18, 19, 36, 37, 200, 1], [0, 5, 77, 128, 64, 511], {}, 0),
    "prompts_128": (L(4, 2, 128, 1), 128, [130, 70, 1], [10, 200, 128], {}, 0),
    "prompts_group1": (L(3, 3, 64, 1), 128, [260, 2, 129], [0, 3, 64], {}, 0),
    "prompts_group6": (L(12, 2, 64, 1), 32, [21, 43, 100], [0, 4, 130], {}, 0),
    "prompts_group7": (L(14, 2, 128, 2), 16, [18, 37, 5], [60, 0, 128], {}, 0),
    "prompts_group8": (L(64, 8, 128, 8), 64, [33, 16, 7], [0, 100, 257], {}, 0),
    "chunk_of_long": (L(8, 2, 128, 2), 64, [70], [4000], {}, 0),
    "chunk_of_long_64": (L(8, 2, 64, 2), 16, [70], [4000], {}, 0),
    "mixed": (QWEN, 32, [1, 300, 1, 1, 40], [2000, 0, 1, 127, 900], {}, 0),
    "sharp": (L(8, 2, 128, 1), 16, [200, 1, 3], [300, 700, 100], dict(sharp=12.0), 0),
    "unlike_scales": (L(8, 2, 128, 1), 16, [200, 1, 3], [300, 700, 100], dict(spread=12, sharp=0.01), 0),
    "far_apart_scales": (L(8, 2, 64, 1), 16, [60, 1, 3], [300, 700, 100], dict(spread=25, sharp=1e-6), 0),
    "rows_behind": (QWEN, 16, [3, 60], [10, 0], dict(extra_rows=77), 0),
    "rows_behind_decode": (QWEN, 16, [1, 1], [10, 0], dict(extra_rows=5), 1),
    "all_empty": (QWEN, 16, [0, 0], [3, 0], dict(extra_rows=9), 0),
    "many_items": (LLAMA, 32, [64] * 20, [100] * 20, {}, 64),
    "few_long_items": (L(8, 2, 64, 1), 128, [128, 90], [2500, 1800], {}, 0),
}


def attend_batch(name, **kw):
    lay, page, new, cached, more, max_new = ATTENDS[name]
    return K.Batch(lay, new, cached, page, **more, **kw), max_new


@pytest.mark.parametrize("name", ATTENDS)
def test_attention(gpu_lib, name):
    import torch
    b, max_new = attend_batch(name)
    d = K.OnDevice(gpu_lib, b, max_new)
    d.attend()
    assert d.status() == 0
    K.check(d.got(), b)
    first = d.out.clone()
    d.out.fill_(7.0)
    d.attend()
    assert torch.equal(first, d.out)


def test_bound_on_new_tokens(gpu_lib):
    b, _ = attend_batch("few_tokens")
    d = K.OnDevice(gpu_lib, b, max_new=2)
    d.attend()
    assert gpu_lib.binding.STATUS_NAMES[d.status()] == "TP_ERR_SHAPE"
    o, bound = b.reference()
    for s, n in enumerate(b.new):
        rows = slice(b.cu[s], b.cu[s] + n)
        got = d.got()[:, rows]
        assert (got == 7.0).all() if n > 2 else (np.abs(got - o[:, rows]) <= bound[:, rows]).all()


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [3, 40, 50, 2]])
def test_rows_outside_the_pages(gpu_lib, new):
    b = K.Batch(L(8, 2, 64, 2), new, [32, 29, -1, 5], 16, width=2)
    d = K.OnDevice(gpu_lib, b)
    d.attend()
    assert gpu_lib.binding.STATUS_NAMES[d.status()] == "TP_ERR_CAPACITY"
    K.check(d.got(), b)


@pytest.mark.parametrize("new", [[1, 1, 1], [30, 3, 60]])
def test_pages_outside_the_pool_are_not_seen(gpu_lib, new):
    b = K.Batch(L(8, 2, 128, 2), new, [40, 9, 100], 16)
    lost = [(0, 1), (1, 0), (2, 0), (2, 3)]
    good = b.table.copy()
    for s, w in lost:
        b.table[s, w] = -1 if w else b.n_pages
    d = K.OnDevice(gpu_lib, b)
    d.attend()
    assert gpu_lib.binding.STATUS_NAMES[d.status()] == "TP_ERR_CAPACITY"
    got = d.got()
    b.table = good
    for r in range(2):
        for s, n in enumerate(new):
            for i in range(n):
                t, p = b.cu[s] + i, b.cached[s] + i
                seen = np.array([(s, j // 16) not in lost for j in range(p + 1)])
                k, v = b.keys("k", s, r, p + 1), b.keys("v", s, r, p + 1)
                for h in range(b.lay.hq):
                    if not seen.any():
                        assert (got[r, t, h] == 0).all()
                        continue
                    x = k[h // b.lay.group][seen] @ b.q[r, t, h] / np.sqrt(128)
                    w = np.exp(x - x.max())
                    want = w @ v[h // b.lay.group][seen] / w.sum()
                    most = np.abs(v[h // b.lay.group][seen]).max()
                    assert (np.abs(got[r, t, h] - want) <= 2.0 ** -7 * most).all()
