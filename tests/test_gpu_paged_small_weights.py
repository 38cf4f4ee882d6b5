"""Attention over 8-bit pages where a page's keys have weights below float32's
smallest number, and its values are as much larger than the others': what counts
is the product, in a row of one piece and in one of many."""
import numpy as np
import pytest

from tests import _paged as K
from tests.test_gpu_paged_unseen import SEEN, attend, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nats,small,large", [(95, -100, 40), (86, -100, 26), (85, -126, 0), (140, -120, 80), (100, -60, 90), (60, -126, -20)])
@pytest.mark.parametrize("name", SEEN)
def test_small_weights_of_large_values(gpu_lib, name, nats, small, large):
    lay, page, new, cached, max_new = SEEN[name]
    b = K.Batch(lay, new, cached, page, spread=0)
    b.q[..., 0] = 16.0
    b.codes["k"][..., 0] &= 0x80
    b.scale["k"][:] = 2.0 ** -9
    b.scale["v"][:] = 2.0 ** small
    for s in range(len(new)):
        at = b.table[s, 1]
        b.codes["k"][:, at] = 0
        b.codes["k"][:, at, :, :, 0] = K.encode(-128.0)
        b.scale["k"][:, at] = np.float32(nats * np.sqrt(lay.d) / 16 / 128)
        b.scale["v"][:, at] = 2.0 ** large
    check(attend(gpu_lib, b, max_new), b)
