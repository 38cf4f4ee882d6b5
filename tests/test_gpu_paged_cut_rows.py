"""Attention over 8-bit pages of values near float32's largest, in rows that are
cut into parts: finite as in one piece."""
import numpy as np
import pytest

from tests import _paged as K

pytestmark = pytest.mark.gpu

L = K.Layout
CUT = {
    "one_row": (L(8, 1, 128, 1), 128, [1], [9000], 1),
    "one_row_64": (L(8, 2, 64, 2), 16, [1, 1], [5000, 300], 1),
    "few_rows": (L(8, 2, 128, 1), 32, [4, 3], [4000, 700], 4),
    "groups_of_rows": (L(8, 1, 64, 1), 16, [3, 4], [3000, 100], 4),
    "prompt": (L(8, 2, 128, 1), 64, [70, 40], [4000, 10], 0),
    "prompt_64": (L(8, 2, 64, 2), 16, [90], [3000], 0),
}


@pytest.mark.parametrize("sharp", [0.01, 3.0])
@pytest.mark.parametrize("name", CUT)
def test_large_values_in_parts(gpu_lib, name, sharp):
    lay, page, new, cached, max_new = CUT[name]
    b = K.Batch(lay, new, cached, page, spread=0, sharp=sharp)
    free = (b.codes["v"] & 127) == 127
    b.codes["v"] = np.where(free, b.codes["v"], (b.codes["v"] & 127).astype(np.uint8))     # of one sign: nothing cancels
    b.scale["v"][:] = 2.0 ** 119
    d = K.OnDevice(gpu_lib, b, max_new)
    d.attend()
    assert d.status() == 0
    K.check(d.got(), b)
