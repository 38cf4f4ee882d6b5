"""Attention of packed batches (with and without a shared prefix) and the
packed prefill block against float64, element by element within the bound that
``tests/_packed.py`` derives."""
import numpy as np
import pytest

import oracle as O
import synth
from tests import _packed as K
from tests import _parity as P
from tests import _oracle_runs as R

pytestmark = pytest.mark.gpu

L = K.Layout
LLAMA, QWEN = L(32, 8, 128, 4), L(14, 2, 64, 2)

# name -> (layout, new tokens, cached tokens, prefix, other arguments)
CASES = {
    # single tokens: nothing cached, one block, block edges, several blocks
    "one_token_empty_cache": (L(8, 2, 128, 2), [1], [0], 0, {}),
    "one_token_edges": (L(8, 2, 128, 2), [1] * 6, [126, 127, 128, 129, 255, 511], 0, {}),
    "one_token_long_cache": (QWEN, [1, 1], [5000, 1], 0, dict(extra_kv=3)),
    # prompts: lengths 0, 1 and around tile and block edges, caches at odd rows
    "prompts_ragged_llama": (LLAMA, [0, 1, 31, 32, 33, 63, 64, 65, 0, 130], [0] * 10, 0, {}),
    "prompts_cached_llama": (LLAMA, [5, 64, 129, 1, 40], [0, 1, 127, 300, 128], 0, dict(extra_kv=70)),
    "prompts_qwen": (QWEN, [18, 19, 36, 37, 200, 1], [0, 5, 77, 128, 64, 511], 0, {}),
    "all_empty_but_one": (QWEN, [0, 0, 3, 0], [9, 0, 4, 2], 0, {}),
    # every group size, both head sizes, every shard count
    "group1_d64_tp1": (L(3, 3, 64, 1), [260, 2, 129], [0, 3, 64], 0, {}),
    "group2_d128_tp1": (L(4, 2, 128, 1), [130, 70], [10, 200], 0, {}),
    "group3_d64_tp2": (L(12, 4, 64, 2), [85, 43, 86], [0, 44, 1], 0, {}),
    "group5_d128_tp1": (L(5, 1, 128, 1), [52, 25, 26, 1], [3, 0, 127, 90], 0, {}),
    "group6_d64_tp1": (L(12, 2, 64, 1), [21, 43, 100], [0, 4, 130], 0, {}),
    "group7_d128_tp2": (L(14, 2, 128, 2), [18, 37, 5], [60, 0, 128], 0, {}),
    "group8_d128_tp8": (L(64, 8, 128, 8), [33, 16, 7], [0, 100, 257], 0, {}),
    # long keys that are split over several parts
    "chunk_of_long": (L(8, 2, 128, 2), [70], [4000], 0, {}),
    "mixed_step": (QWEN, [1, 300, 1, 1, 40], [2000, 0, 1, 127, 900], 0, {}),
    # sharp scores: large growth of a row's maximum from block to block
    "sharp_scores": (L(8, 2, 128, 1), [200, 1], [300, 700], 0, dict(sharp=12.0)),
    # rows behind the last sequence
    "rows_behind": (QWEN, [3, 60], [10, 0], 0, dict(extra_rows=77)),
    # a shared prefix: lengths around block edges, few and many tokens per sequence
    "prefix_one_row": (QWEN, [1, 1, 1], [0, 4, 100], 1, {}),
    "prefix_decode": (LLAMA, [1] * 9, [0, 1, 5, 127, 128, 129, 300, 64, 2], 300, {}),
    "prefix_decode_many": (L(8, 2, 64, 2), [1] * 150, list(range(150)), 129, {}),
    "prefix_few_tokens": (QWEN, [3, 0, 5, 1, 17], [0, 9, 40, 200, 1], 256, {}),
    "prefix_prompts": (LLAMA, [70, 0, 129, 64], [0, 3, 10, 128], 127, {}),
    "prefix_prompts_group1": (L(2, 2, 128, 1), [300, 1, 140], [0, 3, 10], 640, {}),
    "prefix_long_split": (L(8, 2, 128, 1), [1, 2], [10, 1000], 6000, {}),
    "prefix_rows_behind": (QWEN, [1, 2, 1], [3, 0, 50], 200, dict(extra_rows=40)),
    "prefix_empty_sequences_first": (QWEN, [0, 0, 1], [3, 0, 50], 100, {}),
    "prefix_all_empty": (QWEN, [0, 0], [3, 0], 100, dict(extra_rows=9)),
    # how items are cut and dealt out: one row over very many parts, a few items over one round of the SMs, sequences
    # for more than one round of the planning CTA
    "one_token_many_parts": (L(8, 1, 128, 1), [1], [20000], 0, {}),
    "items_just_over_a_round": (LLAMA, [64] * 20, [0] * 20, 640, {}),
    "few_items_of_many_blocks": (L(8, 2, 64, 1), [128, 90], [2500, 1800], 0, {}),
    # single tokens beside a prompt of so many items that they are done as its are, or not quite
    "few_rows_beside_a_prompt": (L(32, 8, 64, 2), [1, 1856, 2, 0, 4, 1], [700, 5, 129, 3, 1000, 0], 0, {}),
    "few_rows_beside_a_prompt_and_a_prefix": (L(32, 8, 64, 2), [1, 1856, 2, 0, 4, 1], [700, 5, 129, 3, 1000, 0], 70, {}),
    "few_rows_beside_a_shorter_prompt": (L(32, 8, 64, 2), [1, 1792, 2, 0, 4, 1], [700, 5, 129, 3, 1000, 0], 0, {}),
    # few rows in all: up to 31 sequences and one more, empty ones between, several tokens, parts
    "few_rows_31": (L(4, 4, 64, 1), [1] * 31, [(67 * i) % 300 for i in range(31)], 0, {}),
    "few_rows_32": (L(4, 4, 64, 1), [1] * 32, [(67 * i) % 300 for i in range(32)], 0, {}),
    "few_rows_31_prefix": (L(2, 2, 128, 2), [1, 0] * 15 + [1], [(67 * i) % 300 for i in range(31)], 390, {}),
    "few_rows_32_prefix": (L(2, 2, 128, 2), [1, 0] * 16, [(67 * i) % 300 for i in range(32)], 390, {}),
    "few_rows_several_tokens": (L(8, 2, 128, 2), [2, 0, 1, 0, 4], [500, 3, 0, 9, 1126], 0, {}),
    "few_rows_several_tokens_prefix": (L(8, 2, 128, 2), [2, 0, 1, 0, 4], [500, 3, 0, 9, 1126], 257, {}),
    "few_rows_group8_parts": (L(8, 1, 64, 1), [1, 0, 3], [9000, 5, 3100], 0, {}),
    "few_rows_group8_parts_prefix": (L(8, 1, 64, 1), [1, 0, 3], [9000, 5, 3100], 5000, {}),
    # every number of rows that an item of few rows can have, beside one another; the last blocks end around TMA boxes
    "rows_of_few_rows_group1": (L(2, 2, 64, 1), list(range(1, 33)) + [3] * 12,
                                [(i * 31 + 1) % 270 for i in range(44)], 0, {}),
    "rows_of_few_rows_group3": (L(6, 2, 128, 2), [1, 2, 3, 4, 5, 6, 7, 8, 9, 10] + [1] * 50,
                                [95, 31, 29, 124, 123, 122, 250, 0, 64, 7] + [16 * i + (i % 3) for i in range(50)], 0, {}),
    "rows_of_few_rows_prefix_edges": (L(4, 1, 128, 1), [1] * 3, [30, 31, 32], 161, {}),
    "parts_and_a_rest": (L(32, 32, 64, 1), [512, 3], [8000, 100], 0, {}),
    "many_sequences": (QWEN, [1] * 1100, [(37 * i) % 150 for i in range(1100)], 0, {}),
    "many_sequences_prefix": (L(4, 1, 64, 1), [i % 3 for i in range(1300)], [(11 * i) % 40 for i in range(1300)], 70, {}),
}


def make(name, seed=1):
    lay, new, cached, prefix, kw = CASES[name]
    return K.Batch(lay, new, cached, prefix=prefix, seed=seed, **kw)


@pytest.mark.parametrize("name", list(CASES))
def test_attention_matches_float64(gpu_lib, name):
    b = make(name)
    d = K.OnDevice(gpu_lib, b, prefix_extra=5 if b.prefix else 0)
    d.run()
    assert d.status() == 0
    share = K.check(d.got(), b)
    print(f"{name}: largest error {share:.2f} of the bound")


@pytest.mark.parametrize("name", ["mixed_step", "prefix_decode", "prefix_prompts", "few_rows_several_tokens",
                                  "few_rows_group8_parts_prefix"])
def test_attention_is_deterministic_and_repeats_on_one_workspace(gpu_lib, name):
    import torch
    d = K.OnDevice(gpu_lib, make(name))
    first = d.run().clone()
    d.ws[256 * 1024:].random_()              # the data regions' contents do not matter, only the control words
    d.tb.tp_workspace_init(d.plan, d.ws, d.nbytes)
    for _ in range(3):
        d.out.fill_(7.0)
        assert torch.equal(d.run(), first)


def test_prefix_of_zero_rows_is_the_packed_call(gpu_lib):
    import torch
    d = K.OnDevice(gpu_lib, make("prompts_qwen"))
    first = d.run().clone()
    d.out.fill_(7.0)
    d.tb.tp_attn_prefix(d.plan, d.q, None, 0, 0, (d.k, d.v), d.cu, d.pos, d.b.B, d.b.T, d.out, d.ws, d.nbytes)
    assert torch.equal(d.out, first)


@pytest.mark.parametrize("what", ["inf", "nan", "lowest"])
@pytest.mark.parametrize("prefix", [0, 200])
def test_what_lies_behind_a_sequence_does_not_reach_it(gpu_lib, what, prefix):
    stale = {"inf": np.inf, "nan": np.nan, "lowest": -3.3895e38}[what]
    b = K.Batch(QWEN, [1, 40, 3], [3, 60, 130], prefix=prefix, seed=3, stale=stale, extra_kv=200)
    d = K.OnDevice(gpu_lib, b)
    d.run()
    K.check(d.got(), b)


@pytest.mark.parametrize("value", [np.inf, np.nan])
@pytest.mark.parametrize("lay", [LLAMA, L(2, 2, 64, 1)])
def test_a_later_tokens_overflow_does_not_reach_earlier_rows(gpu_lib, lay, value):
    # a V entry that overflowed: earlier rows are as without it, the rows that see it carry it
    b = K.Batch(lay, [300, 20], [10, 0], seed=4)
    d = K.OnDevice(gpu_lib, b)
    d.v[0][0, 0, 150, 5] = value
    d.v[0][0, 0, 309, 7] = value
    d.run()
    got = d.got()
    o, bound = b.reference()
    G = lay.group
    seen = np.zeros(o.shape, bool)
    seen[0, 140:300, :G, 5] = True           # position 150 is row 140
    seen[0, 299, :G, 7] = True
    assert not np.isfinite(got[:, :b.used][seen]).any()
    ok = ~seen
    assert (np.abs(got[:, :b.used] - o)[ok] <= bound[ok]).all()


def test_positions_outside_the_cache_give_zeros_and_a_status(gpu_lib):
    tb = gpu_lib
    b = K.Batch(QWEN, [30, 4, 3, 2], [90, 100, -2, 200], seed=5, max_kv=100)
    d = K.OnDevice(tb, b)
    d.run()
    assert d.status() == tb.binding.TP_ERR_CAPACITY
    K.check(d.got(), b)
    b = K.Batch(QWEN, [30, 4, 3, 2], [90, 100, -2, 200], prefix=70, seed=5, max_kv=100)
    d = K.OnDevice(tb, b)
    d.run()
    assert d.status() == tb.binding.TP_ERR_CAPACITY
    K.check(d.got(), b)


@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("cu", [[1, 2, 5], [0, 6, 5], [0, 3, 8], [-1, 3, 5], [0, 9, 5]])
def test_malformed_offsets_write_nothing_and_are_recorded(gpu_lib, cu, prefix):
    import torch
    tb = gpu_lib
    b = K.Batch(QWEN, [3, 4], [4, 0], prefix=prefix, seed=6)
    assert b.T == 7
    d = K.OnDevice(tb, b)
    d.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    d.run()
    assert d.status() == tb.binding.TP_ERR_SHAPE
    assert (d.got() == 7.0).all()


@pytest.mark.parametrize("what", ["inf", "nan", "lowest"])
@pytest.mark.parametrize("prefix", [0, 200])
def test_few_rows_what_lies_behind_a_sequence_does_not_reach_it(gpu_lib, what, prefix):
    stale = {"inf": np.inf, "nan": np.nan, "lowest": -3.3895e38}[what]
    b = K.Batch(QWEN, [1, 0, 2, 1], [3, 5, 130, 700], prefix=prefix, seed=3, stale=stale, extra_kv=200)
    d = K.OnDevice(gpu_lib, b)
    d.run()
    K.check(d.got(), b)


@pytest.mark.parametrize("prefix", [0, 70])
def test_few_rows_positions_outside_the_cache_give_zeros_and_a_status(gpu_lib, prefix):
    tb = gpu_lib
    b = K.Batch(L(8, 2, 128, 1), [3, 2, 1, 1], [98, -1, 99, 200], prefix=prefix, seed=5, max_kv=100)
    d = K.OnDevice(tb, b)
    d.run()
    assert d.status() == tb.binding.TP_ERR_CAPACITY
    K.check(d.got(), b)


@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("cu", [[1, 2, 3], [0, 4, 3], [0, 3, 8], [-1, 2, 3], [0, 9, 3], [0, 2147483647, 3]])
def test_few_rows_malformed_offsets_write_nothing_and_are_recorded(gpu_lib, cu, prefix):
    import torch
    tb = gpu_lib
    b = K.Batch(QWEN, [1, 2], [4, 300], prefix=prefix, seed=6)
    d = K.OnDevice(tb, b)
    d.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    d.run()
    assert d.status() == tb.binding.TP_ERR_SHAPE
    assert (d.got() == 7.0).all()


@pytest.mark.parametrize("prefix", [0, 150])
def test_few_rows_captured_call_replays_with_other_lengths(gpu_lib, prefix):
    import torch
    tb = gpu_lib
    full = K.Batch(QWEN, [2, 1, 1], [900, 900, 900], prefix=prefix, seed=7)
    d = K.OnDevice(tb, full)
    want = d.run().clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.run()
    for new, cached in (([1, 0, 1], [5, 0, 640]), ([0, 0, 4], [1, 1, 127]), ([2, 1, 1], [900, 900, 900])):
        d.cu.copy_(torch.tensor(np.cumsum([0] + new), dtype=torch.int32))
        d.pos.copy_(torch.tensor(cached, dtype=torch.int32))
        d.out.fill_(7.0)
        g.replay()
        replayed = d.out.clone()
        d.out.fill_(7.0)
        assert torch.equal(d.run(), replayed)
        assert (replayed[:, sum(new):] == 7.0).all()
    assert torch.equal(replayed, want)


@pytest.mark.parametrize("prefix", [0, 150])
def test_captured_call_replays_with_other_lengths(gpu_lib, prefix):
    import torch
    tb = gpu_lib
    full = K.Batch(QWEN, [40, 30, 30], [100, 100, 100], prefix=prefix, seed=7)
    d = K.OnDevice(tb, full)
    d.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.run()
    for new, cached in (([40, 30, 30], [100, 100, 100]), ([1, 1, 1], [139, 129, 0]), ([0, 5, 60], [0, 10, 70])):
        b = K.Batch(QWEN, new, cached, prefix=prefix, seed=7, max_kv=full.max_kv, stale=0.0)
        b.T, b.q, b.pk, b.pv = full.T, full.q, full.pk, full.pv
        b.k, b.v = full.k, full.v
        d.cu.copy_(torch.from_numpy(b.cu))
        d.pos.copy_(torch.tensor(cached, dtype=torch.int32))
        d.out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert d.status() == 0
        K.check(d.got(), b)


def test_two_graphs_that_share_a_workspace_replay_in_turn(gpu_lib):
    import torch
    a, c = K.OnDevice(gpu_lib, make("mixed_step")), K.OnDevice(gpu_lib, make("prefix_few_tokens"))
    big = a if a.nbytes >= c.nbytes else c
    a.ws = c.ws = big.ws
    a.run(), c.run()
    refs = (a.out.clone(), c.out.clone())
    torch.cuda.synchronize()
    graphs = []
    for x in (a, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    for _ in range(4):
        for x, g, ref in zip((a, c), graphs, refs):
            x.out.fill_(7.0)
            g.replay()
            assert torch.equal(x.out, ref)


def test_two_streams_with_workspaces_of_their_own(gpu_lib):
    import torch
    ds = [K.OnDevice(gpu_lib, make(n)) for n in ("chunk_of_long", "prefix_decode_many")]
    refs = [d.run().clone() for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                d.out.fill_(7.0)
            d.run(stream=s)
    torch.cuda.synchronize()
    for d, ref in zip(ds, refs):
        assert torch.equal(d.out, ref)


def test_long_cache_past_32_bit_offsets(gpu_lib):
    # one shard's cache holds more than 2^31 elements; the last sequence lies behind them
    import torch
    tb = gpu_lib
    lay, rows, B = L(8, 4, 128, 1), 140000, 32
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB of device memory")
    assert B * lay.hkv * rows * lay.d > 2 ** 31
    k = torch.zeros(B, lay.hkv, rows, lay.d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = K.Batch(lay, [0] * (B - 1) + [3], [0] * (B - 1) + [297], seed=8, stale=0.0)
    for dst, src in ((k, small.k[0]), (v, small.v[0])):
        dst[B - 1, :, :300].copy_(torch.from_numpy(src[B - 1].astype(np.float32)))
    d = K.OnDevice(tb, small)
    plan = tb.tp_plan(K.plan_desc(tb, lay, B, small.T, rows), 1)
    nb = tb.tp_plan_get_info(plan)["workspace_bytes"]
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    tb.tp_workspace_init(plan, ws, nb)
    tb.tp_attn_packed(plan, d.q, ([k], [v]), d.cu, d.pos, B, small.T, d.out, ws, nb)
    assert tb.tp_get_device_status(ws) == 0
    K.check(d.got(), small)


# ---------------------------------------------------------------- the packed block

BLOCKS = {
    "llama_tp2": synth.scaled(synth.WORKLOADS["llama3_8b_prefill_tp8"], hidden=512, n_heads=8, n_kv_heads=2, ffn=1024,
                              tp=2, batch=4, tokens_per_seq=70, kv_len=90, seed=41),
    "qwen_tp2_bias": synth.scaled(synth.WORKLOADS["llama3_8b_prefill_tp8"], hidden=896, n_heads=14, n_kv_heads=2,
                                  head_dim=64, ffn=1152, tp=2, batch=4, tokens_per_seq=70, kv_len=90, qkv_bias=True,
                                  rope_theta=1e6, eps=1e-6, seed=42),
    "hidden_448_tp1": synth.scaled(synth.WORKLOADS["llama3_8b_prefill_tp8"], hidden=448, n_heads=7, n_kv_heads=1,
                                   head_dim=64, ffn=192, tp=1, batch=4, tokens_per_seq=70, kv_len=90, seed=43),
}
TOL = 2e-2                       # as the other blocks: bf16 storage, float32 accumulation, normwise


def block_oracle(inputs, x, new, cached, prefix, pk, pv, k0, v0, max_kv):
    """y rows and the caches after the block, one sequence at a time: the prefix is the first rows of its cache."""
    w = inputs["workload"]
    y = np.zeros((sum(new), w.hidden))
    k1, v1, t = k0.copy(), v0.copy(), 0
    for b, (n, c) in enumerate(zip(new, cached)):
        if n:
            kc = np.concatenate([pk, k0[b]], 1)[None]
            vc = np.concatenate([pv, v0[b]], 1)[None]
            shards = O.shard_layer(O.layer_f64(inputs["layers"][0]), w, w.tp)
            ks, vs = O.shard_kv_cache(kc, w.tp), O.shard_kv_cache(vc, w.tp)
            y[t:t + n] = O.block_tpN(shards, np.asarray(x[t:t + n], np.float64), ks, vs, np.array([prefix + c]), n, w, w.tp)
            k1[b] = np.concatenate(ks, 1)[0][:, prefix:]
            v1[b] = np.concatenate(vs, 1)[0][:, prefix:]
        t += n
    return y, k1, v1


def block_setup(name, prefix, seed=0):
    import torch
    from megatron_tensor_block_gb300.runtime import Model
    w = BLOCKS[name]
    inputs = synth.make_inputs(w, with_head=False)
    m = Model(inputs)
    rng = np.random.default_rng(900 + seed)
    pk, pv = (K.bf16(rng.standard_normal((w.n_kv_heads, prefix, w.head_dim))) for _ in range(2))
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(torch.bfloat16)  # noqa: E731
    per = w.n_kv_heads // w.tp
    pre = ([up(pk[r * per:(r + 1) * per]) for r in range(w.tp)], [up(pv[r * per:(r + 1) * per]) for r in range(w.tp)])
    k0, v0 = (R.full_cache(inputs[n][0], m.max_kv) for n in ("k_cache", "v_cache"))
    return w, inputs, m, pk, pv, pre, k0, v0


@pytest.mark.parametrize("prefix", [0, 130])
@pytest.mark.parametrize("name", list(BLOCKS))
def test_packed_block_matches_oracle(gpu_lib, name, prefix):
    import torch
    w, inputs, m, pk, pv, pre, k0, v0 = block_setup(name, prefix)
    new, cached = [70, 0, 1, 33], [90, 5, 17, 0]
    T = sum(new) + 20
    x = np.asarray(inputs["x"])[:T]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    pos = torch.tensor(cached, dtype=torch.int32, device="cuda")
    xd = torch.from_numpy(np.ascontiguousarray(x)).to("cuda")
    y = torch.full_like(xd, 7.0)
    m.forward_packed(xd, y, cu, pos, [pre] if prefix else None, prefix, prefix)
    assert m.ws.status() == 0
    ref, k1, v1 = block_oracle(inputs, x, new, cached, prefix, pk, pv, k0, v0, m.max_kv)
    got = y.double().cpu().numpy()
    assert P.err(got[:sum(new)], ref) <= TOL
    assert (got[sum(new):] == 7.0).all()
    k, v = (t.double().cpu().numpy() for t in m.caches[0].full())
    for b, (n, c) in enumerate(zip(new, cached)):
        rows = slice(c, c + n)
        if n:
            assert P.err(k[b, :, rows], k1[b, :, rows]) <= TOL and P.err(v[b, :, rows], v1[b, :, rows]) <= TOL
        k[b, :, rows], v[b, :, rows] = k0[b, :, rows], v0[b, :, rows]
    assert np.array_equal(k, k0) and np.array_equal(v, v0)


def test_packed_block_equals_the_prefill_block_on_equal_lengths(gpu_lib):
    # the same projections; the two attention kernels round at the same places, so the blocks agree to rounding
    import torch
    w, inputs, m, *_ = block_setup("llama_tp2", 0)
    y0 = m.forward().clone()
    cu = torch.arange(w.batch + 1, dtype=torch.int32, device="cuda") * w.tokens_per_seq
    y1 = m.forward_packed(m.x, torch.empty_like(m.x), cu, m.pos)
    assert m.ws.status() == 0
    assert P.err(y1.double().cpu().numpy(), y0.double().cpu().numpy()) <= 4e-3


def test_packed_block_reports_capacity_and_malformed_offsets(gpu_lib):
    import torch
    tb = gpu_lib
    w, inputs, m, *_ = block_setup("llama_tp2", 0)
    k_before = [c.clone() for c in m.caches[0].k]
    y = torch.full_like(m.x, 7.0)
    cu = torch.tensor([0, 5, 3, 9, 12], dtype=torch.int32, device="cuda")
    m.forward_packed(m.x, y, cu, m.pos)
    assert m.ws.status() == tb.binding.TP_ERR_SHAPE
    assert (y == 7.0).all() and all(torch.equal(a, b) for a, b in zip(k_before, m.caches[0].k))
    tb.tp_workspace_init(m.plan, m.ws.buf, m.ws.nbytes)
    cu = torch.tensor([0, 5, 9, 9, 12], dtype=torch.int32, device="cuda")
    pos = torch.tensor([m.max_kv - 2, -1, 0, 10], dtype=torch.int32, device="cuda")
    m.forward_packed(m.x, y, cu, pos)
    assert m.ws.status() == tb.binding.TP_ERR_CAPACITY
    assert torch.isfinite(y[:12]).all() and (y[12:] == 7.0).all()


def test_requests_from_prompt_to_constrained_logits(gpu_lib):
    """The operators as a server uses them: unlike prompts behind a shared
    prefix in one packed prefill, a packed decode step, the head, and every
    request's own penalties, biases and grammar."""
    import torch
    tb = gpu_lib
    prefix = 130
    w, inputs, m, pk, pv, pre, k0, v0 = block_setup("llama_tp2", prefix)
    V = 1000
    rng = np.random.default_rng(77)
    head = K.bf16(0.02 * rng.standard_normal((V, w.hidden)))
    gamma = (1 + 0.02 * rng.standard_normal(w.hidden)).astype(np.float32)
    plan = tb.tp_plan(dict(hidden=w.hidden, n_heads=w.n_heads, n_kv_heads=w.n_kv_heads, head_dim=w.head_dim, ffn=w.ffn,
                           n_experts=0, top_k=0, expert_ffn=0, org_vocab=V, eps=w.eps, rope_theta=w.rope_theta,
                           dtype=tb.TP_BF16, has_qkv_bias=0, max_batch=4, max_tokens=280, max_kv=m.max_kv,
                           expert_parallel=0), w.tp)
    info = tb.tp_plan_get_info(plan)
    heads = [torch.empty(info["vocab_rows_shard"], w.hidden, dtype=torch.bfloat16, device="cuda") for _ in range(w.tp)]
    tb.tp_shard_param(plan, tb.TP_PARAM_VOCAB_PARALLEL, torch.from_numpy(head.astype(np.float32)).to("cuda").to(torch.bfloat16),
                      V, w.hidden, tb.TP_BF16, heads)
    new, cached, B = [70, 4, 1, 33], [0, 0, 0, 0], 4
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    x = np.asarray(inputs["x"])[:sum(new)]
    step = np.asarray(inputs["x"])[sum(new):sum(new) + B]
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda")  # noqa: E731
    y = m.forward_packed(up(x), torch.empty(sum(new), w.hidden, device="cuda"), i32([0, 70, 74, 75, 108]), i32(cached),
                         [pre], prefix, prefix)
    z = m.forward_packed(up(step), torch.empty(B, w.hidden, device="cuda"), i32([0, 1, 2, 3, 4]), i32(new), [pre], prefix,
                         prefix)
    assert m.ws.status() == 0
    logits = torch.empty(B, V, device="cuda")
    tb.tp_lm_head_forward(plan, heads, up(gamma), z, B, logits)
    tokens, cu_tokens = [5, 5, 9, 9, 9, 700, 3, 999, 999], [0, 6, 6, 9, 9]
    mask = np.full((1, (V + 31) // 32), 0, np.uint32)
    mask[0, 3] = 0xF0
    out = torch.empty_like(logits)
    tb.tp_logits_process(plan, logits, B, out, tokens=i32(tokens), cu_tokens=i32(cu_tokens), n_prompt=i32([2, 0, 1, 0]),
                         repetition=up([1.5, 1.0, 1.1, 2.0]), presence=up([0.25, 0, 0.5, 1]), frequency=up([0.1, 0, 0, 1]),
                         bias_ids=i32([17]), bias_values=up([100.0]), cu_bias=i32([0, 0, 1, 1, 1]),
                         mask=torch.from_numpy(mask.view(np.int32)).to("cuda"), mask_row=i32([-1, -1, -1, 0]))
    # float64, stage by stage
    y_ref, k1, v1 = block_oracle(inputs, x, new, cached, prefix, pk, pv, k0, v0, m.max_kv)
    z_ref, _, _ = block_oracle(inputs, step, [1] * B, new, prefix, pk, pv, k1, v1, m.max_kv)
    h = z_ref / np.sqrt((z_ref ** 2).mean(-1, keepdims=True) + w.eps) * gamma
    l_ref = h @ head.T
    assert P.err(y.double().cpu().numpy(), y_ref) <= TOL and P.err(z.double().cpu().numpy(), z_ref) <= TOL
    assert P.err(logits.double().cpu().numpy(), l_ref) <= TOL
    l = logits.double().cpu().numpy()
    want = l.copy()
    for t, ids, gen, r, a, f in ((0, {5, 9, 700}, {9: 3, 700: 1}, 1.5, 0.25, 0.1), (2, {3, 999}, {999: 2}, 1.1, 0.5, 0.0)):
        for v in ids:
            want[t, v] = l[t, v] / np.float32(r) if l[t, v] > 0 else l[t, v] * np.float32(r)
        for v, c in gen.items():
            want[t, v] -= np.float32(f) * c + a
    want[1, 17] += 100.0
    want[3, [v for v in range(V) if v not in range(100, 104)]] = -np.inf
    got = out.double().cpu().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(fine, np.isfinite(got)) and np.abs(got - want)[fine].max() <= 1e-5
    assert got[1].argmax() == 17 and 100 <= got[3].argmax() < 104
