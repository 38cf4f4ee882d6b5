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
    "very_many": (L(2, 2, 64, 1), R(), 16, [1, 1, 0, 2] * 320, [(7 * i) % 50 for i in range(1280)], {}),
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


@pytest.mark.parametrize("pos", [5, -7])
@pytest.mark.parametrize("cu", [[0, 5, 3], [1, 3, 6], [0, 3, 99], [0, -1, 6], [-4, 0, 6]])
def test_malformed_offsets_write_nothing(gpu_lib, cu, pos):
    import torch
    b = K.Batch(L(2, 2, 64, 1), [3, 3], [pos, 16], 16)
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
    # a few single tokens that go with a prompt, and more that do not
    "few_beside_a_prompt": (L(32, 8, 64, 2), 64, [1, 600, 2, 0, 4, 1], [700, 5, 129, 3, 1000, 0], {}, 0),
    "many_beside_a_prompt": (L(8, 8, 64, 1), 16, [1] * 40 + [70], [600] * 40 + [10], {}, 0),
    "groups_of_rows": (L(8, 1, 64, 1), 16, [3, 4, 1, 2], [100, 31, 70, 256], {}, 4),
    "groups_of_rows_128": (L(6, 2, 128, 2), 32, [10, 3, 6, 1], [100, 31, 700, 256], {}, 10),
    # more sequences than a CTA has threads
    "very_many": (L(2, 2, 64, 1), 16, [1, 1, 0, 2] * 320, [(7 * i) % 50 for i in range(1280)], {}, 0),
    "very_many_prompts": (L(2, 2, 64, 1), 16, [33, 1, 40, 0] * 150, [(7 * i) % 50 for i in range(600)], {}, 0),
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


def formula(b, r, s, i, h, v=None):
    """Attention of one row in float64, NaN and all."""
    p = b.cached[s] + i
    k = b.keys("k", s, r, p + 1)[h // b.lay.group]
    v = b.keys("v", s, r, p + 1)[h // b.lay.group]
    with np.errstate(invalid="ignore", over="ignore"):
        x = k @ b.q[r, b.cu[s] + i, h] / np.sqrt(b.lay.d)
        w = np.exp(x - x.max())
        return w @ v / w.sum(), np.abs(v).max()


@pytest.mark.parametrize("new", [[1, 1, 1], [4, 2, 3], [9, 40, 150]], ids=["decode", "few", "prompts"])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_reaches_the_rows_that_see_it(gpu_lib, new, d):
    """NaN in a key: every row that sees it, whole. In a value: that feature. In a query: its row. Not elsewhere, and not from
    slots that a row does not see."""
    lay = L(8, 4, d, 2)
    b = K.Batch(lay, new, [40, 130, 5], 16)
    spots = []                                              # (which, shard, kv head, sequence, position, feature)
    for s, n in enumerate(new):
        last = b.cached[s] + n - 1
        spots += [("v", 0, 1, s, last, 3), ("v", 1, 0, s, max(0, last - n // 2), d - 1), ("k", 1, 1, s, last, 0)]
    spots += [("v", 0, 0, 1, 7, 0), ("k", 0, 1, 0, 11, 2)]
    for which, r, kv, s, p, i in spots:
        b.codes[which][r, b.table[s, p // 16], kv, p % 16, i] = 0xFF if i % 2 else 0x7F
    b.q[0, b.cu[1], 2, 5], b.q[1, b.cu[2], 0, 1] = np.inf, np.nan
    dev = K.OnDevice(gpu_lib, b)
    dev.attend()
    assert dev.status() == 0
    got = dev.got()
    for r in range(2):
        for s, n in enumerate(new):
            for i in range(n):
                for h in range(lay.hq):
                    want, most = formula(b, r, s, i, h)
                    if not np.isfinite(b.q[r, b.cu[s] + i, h]).all():
                        want = np.full(d, np.nan)
                    g = got[r, b.cu[s] + i, h]
                    assert (np.isnan(g) == np.isnan(want)).all(), (r, s, i, h, np.argwhere(np.isnan(g) != np.isnan(want))[:4])
                    most = np.nanmax(np.abs(b.keys("v", s, r, b.cached[s] + i + 1)))
                    ok = np.isfinite(want)
                    assert (np.abs(g - want)[ok] <= 2.0 ** -7 * most).all()


@pytest.mark.parametrize("new", [[1, 1], [3, 2], [70, 33]], ids=["decode", "few", "prompts"])
def test_extremes(gpu_lib, new):
    """Zeros, the largest values with the largest scales, and queries of unlike sizes."""
    b = K.Batch(L(8, 2, 64, 1), new, [100, 31], 16, spread=0)
    b.q[0, :, 0], b.q[0, :, 1], b.q[0, :, 2] = 0.0, K.bf16(b.q[0, :, 1] * 1e30), K.bf16(b.q[0, :, 2] * 1e-30)
    b.scale["v"][0, :, 1] = 2.0 ** 110
    b.scale["v"][0, :, 0] = 2.0 ** -60
    b.scale["k"][0, :, 0] = 2.0 ** -60
    d = K.OnDevice(gpu_lib, b)
    d.attend()
    assert d.status() == 0
    K.check(d.got(), b)


def test_two_streams_with_workspaces_of_their_own(gpu_lib):
    import torch
    batches = [attend_batch("mixed"), attend_batch("decode"), attend_batch("prompts_cached")]
    devs = [K.OnDevice(gpu_lib, b, m) for b, m in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in devs]
    for _ in range(5):
        for d, s in zip(devs, streams):
            d.attend(s)
    torch.cuda.synchronize()
    for d in devs:
        assert d.status() == 0
        K.check(d.got(), d.b)


@pytest.mark.parametrize("name,max_new", [("decode", 1), ("mixed", 0), ("few_tokens", 4)])
def test_captured_calls_replay_with_other_lengths(gpu_lib, name, max_new):
    """Append and attend in one graph, two graphs on one workspace; the replays follow what the offsets, positions, table and
    rows hold by then."""
    import torch
    b, _ = attend_batch(name)
    d = K.OnDevice(gpu_lib, b, max_new)
    rope = R(theta=1e4)
    q_out = torch.empty_like(d.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                d.append(rope, q=d.q, q_out=q_out, stream=side)
                gpu_lib.tp_attn_paged(d.plan, q_out, d.kv, d.cu, d.pos, b.B, b.T, d.out, d.ws, d.nbytes, max_new, side)
            graphs.append(g)
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    first = d.out.clone()
    # the sequences in another order, shorter by what the last have more
    order = list(range(b.B))[::-1]
    new, cached = [b.new[i] for i in order], [b.cached[i] for i in order]
    d.cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32))
    d.pos.copy_(torch.tensor(cached, dtype=torch.int32))
    d.table.copy_(d.table.flip(0).clone())
    rows = torch.cat([torch.arange(int(b.cu[i]), int(b.cu[i]) + b.new[i]) for i in order] + [torch.arange(b.used, b.T)]).cuda()
    for x in (d.q, d.new_k, d.new_v):
        x.copy_(x[:, rows].clone())
    graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert d.word.item() == 0 and d.status() == 0
    # the same values, summed up in another order where parts fall differently
    got, want = d.out[:, :b.used].float(), first[:, rows[:b.used]].float()
    assert (got - want).abs().max() <= 2.0 ** -7 * want.abs().max()


def test_chunks_then_single_tokens(gpu_lib):
    """As a server runs them: prompts appended and attended to in chunks, then token by token; every step against float64 over
    the rotated keys and values that the steps before have stored."""
    import torch
    lay, rope, page = L(8, 2, 128, 2), WAVES, 32
    steps = [[50, 7, 33], [30, 0, 1], [1, 1, 1], [2, 1, 0], [1, 3, 1], [1, 1, 1]]
    total = [sum(s[i] for s in steps) for i in range(3)]
    base = K.Batch(lay, total, [0, 0, 0], page)
    base.codes = {n: np.full_like(base.codes[n], 0x7F) for n in "kv"}
    dev = K.OnDevice(gpu_lib, base)
    fed = [0, 0, 0]
    for step, new in enumerate(steps):
        T = sum(new)
        rows = np.concatenate([base.cu[i] + fed[i] + np.arange(n) for i, n in enumerate(new)]).astype(int)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
        pos = torch.tensor(fed, dtype=torch.int32).cuda()
        q, k, v = (x[:, rows].contiguous() for x in (dev.q, dev.new_k, dev.new_v))
        q_out, out = torch.empty_like(q), torch.empty_like(q)
        gpu_lib.tp_kv_append_paged(dev.plan, gpu_lib.tp_rope(**rope), k, v, dev.kv, cu, pos, 3, T, q=q, q_out=q_out,
                                   device_status=dev.word)
        gpu_lib.tp_attn_paged(dev.plan, q_out, dev.kv, cu, pos, 3, T, out, dev.ws, dev.nbytes, max(new))
        now = K.Batch(lay, new, fed, page, width=base.width)
        now.n_pages, now.table = base.n_pages, base.table
        now.q = q_out.double().cpu().numpy()
        now.codes = {n: np.stack([x.cpu().numpy() for x in dev.pool[n]]) for n in "kv"}
        now.scale = {n: np.stack([x.cpu().numpy().astype(np.float64) for x in dev.scale[n]]) for n in "kv"}
        K.check(out.double().cpu().numpy(), now)
        # what is stored stands for the rotated keys: four significant bits, brought to a larger scale at most a few times
        for i, n in enumerate(new):
            fed[i] += n
            for r in range(2):
                at = slice(int(base.cu[i]), int(base.cu[i]) + fed[i])
                want = K.rotate(base.new_k[r, at][None], np.arange(fed[i]), rope, 5e5)[0][0].transpose(1, 0, 2)
                got = now.keys("k", i, r, fed[i])
                e = np.repeat(now.scale["k"][r, now.table[i, :-(-fed[i] // page)]].T, page, 1)[:, :fed[i], None]
                assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) * 1.01 + 2.0 ** -9 * e).all()
    assert dev.word.item() == 0 and dev.status() == 0


@pytest.mark.parametrize("new", [[1, 1], [40, 2]])
def test_pools_beyond_two_to_the_31(gpu_lib, new):
    """Pages whose bytes lie more than 2^31 behind a pool's beginning."""
    import torch
    b = K.Batch(L(4, 1, 128, 1), new, [130, 60], 128)
    far = 140000
    d = K.OnDevice(gpu_lib, b)
    pool = {n: torch.zeros(far + b.n_pages, 1, 128, 128, dtype=torch.uint8, device="cuda") for n in "kv"}
    scale = {n: torch.ones(far + b.n_pages, 1, device="cuda") for n in "kv"}
    for n in "kv":
        pool[n][far:], scale[n][far:] = d.pool[n][0], d.scale[n][0]
    d.kv = gpu_lib.PagedKV(d.plan, [pool["k"]], [pool["v"]], [scale["k"]], [scale["v"]], torch.where(d.table >= 0, d.table + far, -1).to(torch.int32))
    d.attend()
    assert d.status() == 0
    K.check(d.got(), b)
    d.append(R(theta=1e4))
    for n in "kv":
        assert (pool[n][:far].view(torch.int64) == 0).all() and (scale[n][:far] == 1).all()
        d.pool[n], d.scale[n] = [pool[n][far:]], [scale[n][far:]]
    check_pages(d, b, R(theta=1e4))
