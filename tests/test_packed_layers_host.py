"""Model.forward_packed through several layers (no GPU): which buffers the
layers' calls get. The intermediate one must be the model's, not one from the
allocator's pool of the current stream: the layers run on the stream that the
caller names, which does not wait for what that pool's stream still does with
a block's former owner."""
import types

import pytest
import torch

from megatron_tensor_block_gb300 import runtime


@pytest.mark.parametrize("layers", [1, 2, 3, 4])
@pytest.mark.parametrize("rows", [1, 7, 16])
def test_the_layers_pass_through_the_models_own_buffer(monkeypatch, layers, rows):
    calls = []
    monkeypatch.setattr(runtime.B, "tp_block_forward_packed", lambda plan, shards, kv, x, y, *a: calls.append((x, y, a)))
    cache, layer = types.SimpleNamespace(k=[], v=[]), types.SimpleNamespace(shards={})
    m = types.SimpleNamespace(layers=[layer] * layers, caches=[cache] * layers, plan=None, ws=types.SimpleNamespace(buf=0, nbytes=0),
                              tmp=torch.zeros(16, 8) if layers > 1 else None)
    x, y = torch.zeros(rows, 8), torch.zeros(rows, 8)
    cu, pos = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    assert runtime.Model.forward_packed(m, x, y, cu, pos, stream=1234) is y
    assert calls[0][0] is x and calls[-1][1] is y
    for (a, b, rest), after in zip(calls, calls[1:] + [None]):
        assert b.shape == (rows, 8) and b.data_ptr() in (y.data_ptr(), m.tmp.data_ptr() if layers > 1 else 0)
        assert a.data_ptr() != b.data_ptr() and (after is None or after[0] is b)
        assert rest[:4] == (cu, pos, 2, rows) and rest[-1] == 1234
