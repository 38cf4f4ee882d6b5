"""Refusals of the packed block that follow the device check: they name the
call that was made. Nothing is launched."""
import pytest

from tests import _packed as K

pytestmark = pytest.mark.gpu

LAY = K.Layout(14, 2, 64, 2)
A = 1 << 20


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("spoil,status,text", [
    (("wo", 0), "TP_ERR_NULL", "weight pointer is NULL"), (("bqkv", 0), "TP_ERR_NULL", "bias is NULL"),
    (("wgu", A + 8), "TP_ERR_ALIGN", "not 16-byte aligned")])
def test_refusals_name_their_call(gpu_lib, packed, spoil, status, text):
    tb = gpu_lib
    p = tb.tp_plan(K.plan_desc(tb, LAY, 4, 64, 100, has_qkv_bias=1), 2)
    shards = {k: [A, A] for k in ("wqkv", "bqkv", "wo", "wgu", "wd", "gamma_attn", "gamma_ffn")}
    shards[spoil[0]] = [A, spoil[1]]
    kv = ([A, A], [A, A])
    with pytest.raises(tb.TpError) as e:
        if packed:
            tb.tp_block_forward_packed(p, shards, kv, A, 2 * A, A, A, 4, 64, A, p.workspace_bytes, stream=0)
        else:
            tb.tp_block_forward(p, shards, kv, A, 2 * A, A, 4, 16, tb.TP_MODE_PREFILL, None, A, p.workspace_bytes, stream=0)
    who = "tp_block_forward_packed: " if packed else "tp_block_forward: "
    assert str(e.value).startswith(f"{status}: {who}shard 1") and text in str(e.value)
