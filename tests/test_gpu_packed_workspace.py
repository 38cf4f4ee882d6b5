"""The packed calls on workspaces of both layouts: partial results in a place
of their own, or where the prefill buffers lie that no attention stage needs."""
import numpy as np
import pytest

import synth
from tests.test_gpu_packed import BLOCKS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [0, 700])
def test_the_block_gives_the_same_bits_wherever_its_partial_results_lie(gpu_lib, prefix):
    import torch
    from megatron_tensor_block_gb300.runtime import Model, desc_of
    tb = gpu_lib
    w = synth.scaled(BLOCKS["llama_tp2"], ffn=8192, tokens_per_seq=70, kv_len=2500, seed=46)
    m = Model(synth.make_inputs(w, with_head=False))
    new, cached = [1, 0, 40, 2], [2400, 5, 1700, 0]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, pos, T = i32(np.cumsum([0] + new).tolist()), i32(cached), sum(new)
    g = torch.Generator(device="cuda").manual_seed(47)
    pre = [[torch.randn(w.n_kv_heads // w.tp, prefix, w.head_dim, generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(w.tp)] for _ in range(2)]
    outs = []
    kv = (m.caches[0].k, m.caches[0].v)
    for max_tokens in (w.tokens, 20000):
        p = tb.tp_plan(desc_of(w, max_kv=m.max_kv, max_tokens=max_tokens), w.tp)
        ws = torch.full((p.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN wherever it is read unwritten
        tb.tp_workspace_init(p, ws, p.workspace_bytes)
        y = torch.empty(T, w.hidden, device="cuda")
        for _ in range(2):
            tb.tp_block_forward_packed(p, m.layers[0].shards, kv, m.x, y, cu, pos, 4, T, ws, p.workspace_bytes,
                                       pre if prefix else None, prefix, prefix)
        assert tb.tp_get_device_status(ws) == 0
        assert torch.isfinite(y).all()
        outs.append(y)
    # a token's 2 x 8 x 128 x 4 bytes of partial results fit into the 4 x 512 of h and the 2 x 8192 of the SwiGLU output, and
    # with 20000 tokens so do the additional parts'
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("name", ["llama3_8b_decode_tp4", "prefill"])
def test_other_calls_write_nothing_behind_a_workspace_without_the_packed_scratch(gpu_lib, name):
    import torch
    from megatron_tensor_block_gb300.runtime import Model
    tb = gpu_lib
    w = synth.WORKLOADS.get(name) or synth.scaled(BLOCKS["llama_tp2"], kv_len=0, seed=48)
    m = Model(synth.make_inputs(w, with_head=False))
    want = m.forward().clone()

    def taken(n):
        try:
            tb.tp_workspace_init(m.plan, m.ws.buf, n)
            return True
        except tb.TpError:
            return False
    lo, hi = 0, m.ws.nbytes                      # the smallest size that is taken
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (lo, mid) if taken(mid) else (mid, hi)
    assert hi < m.ws.nbytes
    m.ws.buf, m.ws.nbytes = torch.full((hi + 4096,), 0xA5, dtype=torch.uint8, device="cuda"), hi
    tb.tp_workspace_init(m.plan, m.ws.buf, hi)
    assert torch.equal(m.forward(), want)
    assert m.ws.status() == 0 and (m.ws.buf[hi:] == 0xA5).all()
