"""Scales of pages of values, in the attention over 8-bit pages: those that a row
does not see never reach it, and those that it sees count by its weights."""
import numpy as np
import pytest

from tests import _paged as K
from tests import _paged_seen as S

pytestmark = pytest.mark.gpu

L = K.Layout


def check(got, b):
    o, bound = S.reference(b)
    g = got[:, :b.used]
    assert np.isfinite(g).all()
    diff = np.abs(g - o)
    assert (diff <= bound).all(), (float((diff / bound).max()), np.argwhere(diff > bound)[:5].tolist())


def attend(gpu_lib, b, max_new):
    d = K.OnDevice(gpu_lib, b, max_new)
    d.attend()
    assert d.status() == 0
    return d.got()


# new tokens that cross the beginning of a page: (layout, page, new, cached, max_new)
CROSS = {
    "few_64": (L(8, 2, 64, 1), 16, [4, 2, 3], [14, 31, 77], 4),
    "few_128": (L(8, 2, 128, 2), 16, [4, 2, 3], [14, 47, 79], 4),
    "two_groups": (L(8, 1, 64, 1), 16, [4, 3, 1], [13, 46, 15], 4),
    "pages_of_32": (L(8, 2, 128, 1), 32, [4, 2, 3], [30, 63, 127], 4),
    "prompts_16": (L(8, 2, 64, 1), 16, [40, 33, 65], [0, 100, 700], 0),
    "prompts_32_128": (L(8, 2, 128, 2), 32, [40, 70], [10, 300], 0),
    "prompts_64": (L(14, 2, 64, 2), 64, [100, 19], [0, 50], 0),
    "prompt_cut": (L(4, 1, 128, 1), 16, [50], [3000], 0),
}


@pytest.mark.parametrize("by", [15, 26, 30, 60, 100])
@pytest.mark.parametrize("name", CROSS)
def test_unseen_scales(gpu_lib, name, by):
    """The last page's values grow by 2^by: rows before it are the same to the bit, those in it within the bound."""
    lay, page, new, cached, max_new = CROSS[name]
    b = K.Batch(lay, new, cached, page, spread=1)
    first = attend(gpu_lib, b, max_new)
    check(first, b)
    before = np.zeros(b.used, bool)
    for s, (n, c) in enumerate(zip(new, cached)):
        w = (c + n - 1) // page
        b.scale["v"][:, b.table[s, w]] *= 2.0 ** by
        before[b.cu[s]:b.cu[s + 1]] = c + np.arange(n) < w * page
    assert before.any()
    got = attend(gpu_lib, b, max_new)
    assert (got[:, :b.used][:, before] == first[:, :b.used][:, before]).all()
    check(got, b)


SEEN = {
    "one_token": (L(8, 2, 128, 1), 16, [1, 1], [500, 60], 1),
    "one_token_64": (L(4, 2, 64, 2), 64, [1, 1], [500, 200], 1),
    "one_token_cut": (L(2, 1, 64, 1), 128, [1], [20000], 1),
    "few": (L(8, 2, 64, 1), 32, [4, 3], [500, 70], 4),
    "prompts": (L(8, 2, 128, 1), 16, [70, 40], [500, 300], 0),
    "prompts_64": (L(4, 2, 64, 2), 64, [130, 70], [500, 100], 0),
    "prompt_cut": (L(4, 1, 128, 1), 128, [50], [3000], 0),
}


@pytest.mark.parametrize("by", [14, 20, 24, 40, 90])
@pytest.mark.parametrize("name", SEEN)
def test_seen_scales_without_weight(gpu_lib, name, by):
    """A page of large values whose keys every row's softmax leaves out: e^-(2 by)."""
    lay, page, new, cached, max_new = SEEN[name]
    b = K.Batch(lay, new, cached, page, spread=1)
    b.q[..., 0] = 16.0
    for s in range(len(new)):
        at = b.table[s, 1]
        b.codes["k"][:, at, :, :, 0] = K.encode(-224.0)
        b.scale["k"][:, at] = K.bf16(2 * by * np.sqrt(lay.d) / 16 / 224)       # (no power of two)
        b.scale["v"][:, at] *= 2.0 ** by
    check(attend(gpu_lib, b, max_new), b)


@pytest.mark.parametrize("name", SEEN)
def test_values_beyond_float32_without_weight(gpu_lib, name):
    """A page of values of up to 2^129 whose keys have weights of e^-250: parts that hold nothing else are no infinities."""
    lay, page, new, cached, max_new = SEEN[name]
    b = K.Batch(lay, new, cached, page, spread=0)
    b.q[..., 0] = 16.0
    for s in range(len(new)):
        at = b.table[s, 1]
        b.codes["k"][:, at] = 0
        b.codes["k"][:, at, :, :, 0] = K.encode(-250.0)
        b.scale["k"][:, at] = np.float32(np.sqrt(lay.d) / 16)
        b.scale["v"][:, at] = 2.0 ** 121
    check(attend(gpu_lib, b, max_new), b)


@pytest.mark.parametrize("spread", [8, 25, 50])
@pytest.mark.parametrize("name", SEEN)
def test_seen_scales_far_apart(gpu_lib, name, spread):
    lay, page, new, cached, max_new = SEEN[name]
    b = K.Batch(lay, new, cached, page, spread=spread, sharp=0.5)
    b.scale["k"][:] = 1 / 256
    check(attend(gpu_lib, b, max_new), b)


@pytest.mark.parametrize("name", SEEN)
def test_scales_that_are_no_powers_of_two(gpu_lib, name):
    lay, page, new, cached, max_new = SEEN[name]
    b = K.Batch(lay, new, cached, page, spread=3)
    for n in "kv":
        b.scale[n] = (b.scale[n] * b.rng.uniform(0.5, 1.0, b.scale[n].shape)).astype(np.float32).astype(np.float64)
    check(attend(gpu_lib, b, max_new), b)


@pytest.mark.parametrize("name", SEEN)
def test_scales_at_the_ends(gpu_lib, name):
    """Pages of float32's smallest and largest normal scales beside one another."""
    lay, page, new, cached, max_new = SEEN[name]
    b = K.Batch(lay, new, cached, page, spread=0)
    for s in range(len(new)):
        b.scale["v"][:, b.table[s, 0]] = 2.0 ** -126
        b.scale["v"][:, b.table[s, 2]] = 2.0 ** 118
    check(attend(gpu_lib, b, max_new), b)
