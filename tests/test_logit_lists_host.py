"""Lengths of the logit controls' lists: refusals (no GPU). The addresses are
made up; each refusal precedes any launch."""
import pytest

import megatron_tensor_block_gb300 as tb
from megatron_tensor_block_gb300 import binding as B
from tests import _packed as K

A = 1 << 20


def plan():
    return tb.tp_plan(K.plan_desc(tb, K.Layout(14, 2, 64, 2), 4, 64, 100, org_vocab=1000), 2)


@pytest.mark.parametrize("kw", [
    dict(tokens=A, cu_tokens=A), dict(tokens=A, cu_tokens=A, n_tokens=0), dict(tokens=A, cu_tokens=A, n_tokens=-1),
    dict(bias_ids=A, bias_values=A, cu_bias=A), dict(bias_ids=A, bias_values=A, cu_bias=A, n_bias=-5),
    dict(tokens=A, cu_tokens=A, n_tokens=9, bias_ids=A, bias_values=A, cu_bias=A, n_bias=0)])
def test_a_list_without_its_length_is_refused(kw):
    with pytest.raises(tb.TpError) as e:
        tb.tp_logits_process(plan(), A, 2, 2 * A, stream=0, **kw)
    assert e.value.status == B.TP_ERR_SHAPE, str(e.value)


@pytest.mark.parametrize("mask_row", [None, A])
def test_the_address_of_a_mask_needs_its_rows(mask_row):
    # with 0 rows every mask_row would lie outside, and no grammar apply
    with pytest.raises(ValueError, match="mask_rows"):
        tb.tp_logits_process(plan(), A, 2, 2 * A, stream=0, mask=A, mask_row=mask_row)
