"""A packed batch through several layers, on the current and on another
stream, against the float64 oracle layer by layer."""
import numpy as np
import pytest

import synth
from tests import _oracle_runs as R
from tests import _packed as K
from tests import _parity as P
from tests.test_gpu_packed import BLOCKS, TOL, block_oracle

pytestmark = pytest.mark.gpu

NEW, CACHED = [40, 0, 1, 23], [20, 5, 17, 0]


def setup(layers, prefix):
    import torch
    from megatron_tensor_block_gb300.runtime import Model
    w = synth.scaled(BLOCKS["llama_tp2"], n_layers=layers, seed=44)
    inputs = synth.make_inputs(w, with_head=False)
    m = Model(inputs)
    rng = np.random.default_rng(45)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(torch.bfloat16)  # noqa: E731
    per, pre, host = w.n_kv_heads // w.tp, [], []
    for _ in range(layers):
        pk, pv = (K.bf16(rng.standard_normal((w.n_kv_heads, prefix, w.head_dim))) for _ in range(2))
        host.append((pk, pv))
        pre.append(tuple([up(p[r * per:(r + 1) * per]) for r in range(w.tp)] for p in (pk, pv)))
    ref = np.asarray(inputs["x"])[:sum(NEW)]
    for i in range(layers):
        k0, v0 = (R.full_cache(inputs[n][i], m.max_kv) for n in ("k_cache", "v_cache"))
        one = dict(inputs, layers=[inputs["layers"][i]])
        ref, _, _ = block_oracle(one, ref, NEW, CACHED, prefix, *host[i], k0, v0, m.max_kv)
    return w, inputs, m, pre if prefix else None, ref


def batch(inputs):
    import torch
    x = torch.from_numpy(np.ascontiguousarray(np.asarray(inputs["x"])[:sum(NEW)])).to("cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(NEW)]), dtype=torch.int32, device="cuda")
    return x, cu, torch.tensor(CACHED, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("prefix", [0, 130])
@pytest.mark.parametrize("layers", [2, 3])
def test_layers_match_the_oracle(gpu_lib, layers, prefix):
    import torch
    w, inputs, m, pre, ref = setup(layers, prefix)
    x, cu, pos = batch(inputs)
    y = m.forward_packed(x, torch.empty_like(x), cu, pos, pre, prefix, prefix)
    assert m.ws.status() == 0
    assert P.err(y.double().cpu().numpy(), ref) <= TOL


@pytest.mark.parametrize("as_address", [False, True])
def test_layers_on_another_stream_beside_work_of_the_current_one(gpu_lib, as_address):
    # the current stream still writes a block of the output's size that its owner has given back
    import torch
    w, inputs, m, pre, ref = setup(2, 0)
    x, cu, pos = batch(inputs)
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.ones(1 << 28, device="cuda")
    given_back = torch.empty_like(x)
    for _ in range(20):
        big.mul_(1.0)                            # some milliseconds
    given_back.fill_(float("nan"))
    del given_back
    m.forward_packed(x, y, cu, pos, stream=s.cuda_stream if as_address else s)
    torch.cuda.synchronize()
    assert m.ws.status() == 0
    assert P.err(y.double().cpu().numpy(), ref) <= TOL


@pytest.mark.parametrize("layers", [1, 2, 3])
def test_more_rows_than_the_plan_has_are_refused_by_every_number_of_layers(gpu_lib, layers):
    import torch
    from megatron_tensor_block_gb300.runtime import Model
    w = synth.scaled(BLOCKS["llama_tp2"], n_layers=layers, seed=44)
    m = Model(synth.make_inputs(w, with_head=False))
    x = torch.zeros(w.tokens + 1, w.hidden, device="cuda")
    y = torch.full_like(x, 7.0)
    cu = torch.tensor([0, w.tokens + 1], dtype=torch.int32, device="cuda")
    with pytest.raises(gpu_lib.TpError, match="TP_ERR_SHAPE"):
        m.forward_packed(x, y, cu, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert (y == 7.0).all() and m.ws.status() == 0


@pytest.mark.parametrize("prefix", [0, 130])
def test_a_captured_pass_replays_with_other_lengths_in_a_padded_batch(gpu_lib, prefix):
    # rows behind the last sequence hold NaN: they reach nothing and stay as they are
    import torch
    w, inputs, m, pre, _ = setup(2, prefix)
    x = torch.from_numpy(np.ascontiguousarray(np.asarray(inputs["x"])[:90])).to("cuda")
    y = torch.full_like(x, 7.0)
    cu = torch.tensor([0, 40, 60, 70, 80], dtype=torch.int32, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    caches = [[t.clone() for t in c.k + c.v] for c in m.caches]

    def restore():
        for c, old in zip(m.caches, caches):
            for t, o in zip(c.k + c.v, old):
                t.copy_(o)
    m.forward_packed(x, y, cu, pos, pre, prefix, prefix)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.forward_packed(x, y, cu, pos, pre, prefix, prefix)
    for new, cached in (([40, 0, 1, 23], [20, 5, 17, 0]), ([1, 1, 1, 1], [89, 0, 63, 64]), ([0, 0, 0, 70], [0, 0, 0, 90]), ([0] * 4, [0] * 4)):
        n = sum(new)
        cu.copy_(torch.from_numpy(np.cumsum([0] + new).astype(np.int32)))
        pos.copy_(torch.tensor(cached, dtype=torch.int32))
        x.copy_(torch.from_numpy(np.ascontiguousarray(np.asarray(inputs["x"])[:90])))
        x[n:] = float("nan")
        outs = []
        for run in (g.replay, lambda: m.forward_packed(x, y, cu, pos, pre, prefix, prefix),
                    lambda: m.forward_packed(x[:n].contiguous(), y[:n], cu, pos, pre, prefix, prefix)):
            if n == 0 and len(outs) == 2:
                break
            restore()
            y.fill_(7.0)
            run()
            outs.append(y.clone())
        assert m.ws.status() == 0
        assert torch.isfinite(outs[0]).all() and (outs[0][n:] == 7.0).all()
        assert torch.equal(outs[0], outs[1])
        if n:                                           # without the rows behind: other parts, so equal to a rounding
            assert P.err(outs[2][:n].double().cpu().numpy(), outs[0][:n].double().cpu().numpy()) <= TOL
