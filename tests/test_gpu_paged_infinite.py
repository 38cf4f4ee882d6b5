"""Attention over 8-bit pages of rows whose visible scores are all -inf, from an
infinite query or from scores beyond float32: 0 / 0, NaN, in however many parts
the row is. Zeros are for rows that see no key."""
import numpy as np
import pytest

from tests import _paged as K
from tests.test_gpu_paged import formula

pytestmark = pytest.mark.gpu

MINUS_ONE = 0xB8                          # -1 as e4m3
NEW = {"one": [1, 1, 1], "few": [3, 4, 2], "prompts": [40, 70, 33]}


def run(gpu_lib, b):
    d = K.OnDevice(gpu_lib, b)
    d.attend()
    return d


def check_rows(got, b, lost):
    """Rows (shard, token row, head) of `lost` are NaN, the others as the formula has them."""
    for r in range(b.lay.tp):
        for s, n in enumerate(b.new):
            for i in range(n):
                for h in range(b.lay.hq):
                    g = got[r, b.cu[s] + i, h]
                    if (r, b.cu[s] + i, h) in lost:
                        assert np.isnan(g).all(), (r, s, i, h)
                        continue
                    want, most = formula(b, r, s, i, h)
                    assert (np.abs(g - want) <= 2.0 ** -7 * most).all(), (r, s, i, h)


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("d", [64, 128])
def test_an_infinite_query_over_keys_of_one_sign(gpu_lib, new, d):
    b = K.Batch(K.Layout(8, 4, d, 2), NEW[new], [0, 700, 5], 16)
    b.codes["k"][0, :, 1, :, 3] = np.where(b.codes["k"][0, :, 1, :, 3] == 0x7F, 0x7F, MINUS_ONE)
    lost = set()
    for s, h in ((0, 2), (1, 3), (2, 2)):
        for i in {0, b.new[s] - 1}:
            b.q[0, b.cu[s] + i, h, 3] = np.inf
            lost.add((0, b.cu[s] + i, h))
    d = run(gpu_lib, b)
    assert d.status() == 0
    check_rows(d.got(), b, lost)


@pytest.mark.parametrize("new", NEW)
def test_scores_below_float32(gpu_lib, new):
    b = K.Batch(K.Layout(8, 2, 64, 2), NEW[new], [0, 700, 5], 16)
    b.codes["k"][1, :, 0] = np.where(b.codes["k"][1, :, 0] == 0x7F, 0x7F, MINUS_ONE)
    b.scale["k"][1, :, 0] = 2.0 ** 60
    lost = set()
    for s, n in enumerate(b.new):
        for h in range(b.lay.group):
            b.q[1, b.cu[s]:b.cu[s] + n, h] = 2.0 ** 100
            lost |= {(1, b.cu[s] + i, h) for i in range(n)}
    d = run(gpu_lib, b)
    assert d.status() == 0
    check_rows(d.got(), b, lost)


@pytest.mark.parametrize("new", [[1, 1], [4, 3], [64, 40]])
def test_scores_below_float32_beside_others(gpu_lib, new):
    """A page's scores are -inf, those of the others are not: its keys have no weight, wherever the row is cut."""
    b = K.Batch(K.Layout(8, 2, 64, 1), new, [20000, 45], 16)
    for s, w in ((0, 0), (0, 200), (0, 1240), (1, 1)):
        at = b.table[s, w]
        b.codes["k"][0, at, 0] = MINUS_ONE
        b.scale["k"][0, at, 0] = 2.0 ** 120
    b.q[0, :, 0] = np.abs(b.q[0, :, 0]) * 2.0 ** 10
    d = run(gpu_lib, b)
    assert d.status() == 0
    check_rows(d.got(), b, set())


@pytest.mark.parametrize("new", [[1, 1], [40, 60]])
def test_rows_without_keys_stay_zeros(gpu_lib, new):
    """Beside rows that are 0 / 0: where no page is there, an infinite query's row is zeros."""
    b = K.Batch(K.Layout(4, 2, 64, 1), new, [20, 20], 32)
    b.table[0] = -1
    b.codes["k"][0, :, 0, :, 3] = np.where(b.codes["k"][0, :, 0, :, 3] == 0x7F, 0x7F, MINUS_ONE)
    b.q[0, :, 0, 3] = np.inf
    d = run(gpu_lib, b)
    assert gpu_lib.binding.STATUS_NAMES[d.status()] == "TP_ERR_CAPACITY"
    got = d.got()
    assert (got[:, :new[0]] == 0).all()
    assert np.isnan(got[0, new[0]:, 0]).all() and np.isfinite(got[0, new[0]:, 1:]).all()
