"""Appending keys near bf16's largest with a large factor of the rotation: the
scale that they ask for lies beyond float32, and ends at 2^127."""
import numpy as np
import pytest

from tests import _paged as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("factor", [300.0, 2000.0, 1e6])
def test_scales_end_at_the_largest_power(gpu_lib, factor):
    rope = K.rope_args(theta=1e4, attn_factor=factor)
    b = K.Batch(K.Layout(2, 2, 64, 1), [20, 3], [5, 16], 16)
    b.new_k[0, :, 0] = K.bf16(np.sign(b.new_k[0, :, 0]) * 3e38)
    held = b.codes["k"].copy()
    b.scale["k"][:, b.table[0, 0]] = 2.0 ** 125                        # what the first page holds counts beside them
    before = b.scale["k"].copy()
    d = K.OnDevice(gpu_lib, b)
    d.append(rope)
    assert d.word.item() == 0
    got, scale = d.pool["k"][0].cpu().numpy(), d.scale["k"][0].cpu().numpy().astype(np.float64)
    turned, err = K.rotate(b.new_k, b.positions(), rope, 5e5)
    for s in range(2):
        for i in range(b.new[s]):
            p = b.cached[s] + i
            at, t = b.table[s, p // 16], b.cu[s] + i
            assert scale[at, 0] == 2.0 ** 127
            y, e = turned[0, t, 0] / 2.0 ** 127, err[0, t, 0] / 2.0 ** 127
            want = np.clip(y, -448, 448)
            assert (np.abs(K.DECODE[got[at, 0, p % 16]] - want) <= np.where(np.abs(y) > 448 + e, 0, K.half_step(want) + e)).all()
            # the other head's keys are ordinary
            z, e = turned[0, t, 1], err[0, t, 1]
            assert (np.abs(K.DECODE[got[at, 1, p % 16]] * scale[at, 1] - z) <= K.half_step(z / scale[at, 1]) * scale[at, 1] + e).all()
    at = b.table[0, 0]
    kept = K.encode(K.DECODE[held[0, at, 0, :5]] * before[0, at, 0] / 2.0 ** 127)
    assert (got[at, 0, :5] == kept).all()
