"""Offsets of a packed batch whose differences wrap around in 32 bits, in the
attention over 8-bit pages: malformed like any others."""
import pytest

from tests import _paged as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu", [[0, 5, -2 ** 31], [0, 5, 2 - 2 ** 31], [0, 2 ** 31 - 1, 6], [0, 2 ** 31 - 1, -2 ** 31]])
@pytest.mark.parametrize("max_new", [0, 4])
def test_offsets_that_wrap_write_nothing(gpu_lib, cu, max_new):
    import torch
    b = K.Batch(K.Layout(16, 2, 64, 1), [5, 20], [5, 16], 16)
    d = K.OnDevice(gpu_lib, b, max_new)
    d.cu.copy_(torch.tensor(cu))
    d.attend()
    assert gpu_lib.binding.STATUS_NAMES[d.status()] == "TP_ERR_SHAPE"
    assert (d.out == 7).all()
