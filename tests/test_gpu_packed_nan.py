"""A NaN that a row of packed attention sees is a NaN of its results, in
whatever form the row is computed: in one piece, in parts that are joined,
behind a shared prefix, on the path for few rows. Rows that do not see it
stay within the bound of ``tests/_packed.py``."""
import numpy as np
import pytest

from tests import _packed as K

pytestmark = pytest.mark.gpu

L = K.Layout

# name -> (layout, new, cached, prefix)
FORMS = {
    "whole_wide": (L(8, 2, 128, 2), [70, 40], [20, 3], 0),
    "whole_narrow": (L(8, 2, 64, 1), [3, 1, 2] + [1] * 40, [20, 3, 9] + [5] * 40, 0),
    "wide_parts": (L(8, 2, 128, 2), [70], [3000], 0),
    "narrow_parts": (L(4, 1, 64, 1), [1] * 40, [700 + 50 * i for i in range(40)], 0),
    "shared_prefix": (L(32, 8, 128, 4), [1] * 9, [0, 1, 5, 127, 128, 129, 300, 64, 2], 300),
    "shared_long_prefix": (L(8, 2, 64, 1), [1] * 40, [3 * i for i in range(40)], 3000),
    "prefix_of_prompts": (L(4, 2, 128, 1), [200, 129, 90], [0, 3, 10], 127),
    "few_rows": (L(8, 2, 128, 2), [2, 0, 1, 0, 4], [500, 3, 0, 9, 1126], 0),
    "few_rows_one_block": (L(8, 2, 128, 2), [1, 2], [3, 60], 0),
    "few_rows_prefix": (L(8, 2, 128, 2), [2, 0, 1, 0, 4], [500, 3, 0, 9, 1126], 257),
}


def run(tb, b, spoil):
    d = K.OnDevice(tb, b)
    spoil(d)
    d.run()
    assert d.status() == 0
    return d.got()[:, :b.used]


def compare(b, got, nan):
    o, bound = b.reference()
    assert np.isnan(got[nan]).all(), f"{int((~np.isnan(got[nan])).sum())} of {nan.sum()} values are not NaN"
    ok = ~nan
    assert (np.abs(got[ok] - o[ok]) <= bound[ok]).all()


@pytest.mark.parametrize("form", list(FORMS))
def test_a_query_of_nan_gives_nan(gpu_lib, form):
    lay, new, cached, prefix = FORMS[form]
    b = K.Batch(lay, new, cached, prefix=prefix, seed=31)
    t, r, h = b.used - 1, lay.tp - 1, lay.hq - 1

    def spoil(d):
        d.q[r, t, h] = float("nan")
        d.q[0, 0, 0, 5] = float("nan")
    nan = np.zeros((lay.tp, b.used, lay.hq, lay.d), bool)
    nan[r, t, h] = nan[0, 0, 0] = True
    compare(b, run(gpu_lib, b, spoil), nan)


@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("form", list(FORMS))
def test_a_visible_key_of_nan_gives_nan_to_the_rows_that_see_it(gpu_lib, form, where):
    lay, new, cached, prefix = FORMS[form]
    b = K.Batch(lay, new, cached, prefix=prefix, seed=32)
    s = max(i for i in range(b.B) if new[i])
    key = 0 if where == "first" else cached[s] + new[s] - 1

    def spoil(d):
        d.k[0][s, 0, key, 3] = float("nan")
    nan = np.zeros((lay.tp, b.used, lay.hq, lay.d), bool)
    first = int(b.cu[s]) + max(0, key - cached[s])
    nan[0, first:int(b.cu[s + 1]), :lay.group] = True
    compare(b, run(gpu_lib, b, spoil), nan)


@pytest.mark.parametrize("form", ["wide_parts", "narrow_parts", "few_rows"])
def test_a_part_of_nothing_but_nan_is_not_passed_over(gpu_lib, form):
    # every key of the first 256 rows, so that at least a part's first block has no other score
    lay, new, cached, prefix = FORMS[form]
    b = K.Batch(lay, new, cached, prefix=prefix, seed=33)
    s = max(range(b.B), key=lambda i: cached[i])

    def spoil(d):
        d.k[0][s, 0, :256] = float("nan")
    nan = np.zeros((lay.tp, b.used, lay.hq, lay.d), bool)
    nan[0, int(b.cu[s]):int(b.cu[s + 1]), :lay.group] = True
    compare(b, run(gpu_lib, b, spoil), nan)


@pytest.mark.parametrize("form", ["shared_prefix", "shared_long_prefix", "prefix_of_prompts", "few_rows_prefix"])
def test_a_key_of_nan_in_the_prefix_reaches_every_row(gpu_lib, form):
    lay, new, cached, prefix = FORMS[form]
    b = K.Batch(lay, new, cached, prefix=prefix, seed=34)

    def spoil(d):
        d.pk[0][0, prefix - 1, 0] = float("nan")
    nan = np.zeros((lay.tp, b.used, lay.hq, lay.d), bool)
    nan[0, :, :lay.group] = True
    compare(b, run(gpu_lib, b, spoil), nan)


@pytest.mark.parametrize("form", ["wide_parts", "narrow_parts", "shared_prefix", "few_rows_prefix"])
def test_a_value_of_nan_reaches_a_row_that_hardly_weighs_it(gpu_lib, form):
    # Key 0 scores so low that its part's weight is 0 in float32: 0 * NaN is NaN all the same. q = 8 in one dimension, where
    # that key (and with it its part: its other keys as well) has -2^10 and the rest 0: a score of -2^13 / sqrt(d).
    lay, new, cached, prefix = FORMS[form]
    b = K.Batch(lay, new, cached, prefix=prefix, seed=35)
    b.q[:, :, :, 0] = 8.0
    b.k[..., 0] = np.where(np.isnan(b.k[..., 0]), np.nan, 0.0)
    s = max(range(b.B), key=lambda i: cached[i])
    far = (b.pk[0, 0] if prefix else b.k[0, s, 0])[:256]
    b.pk[..., 0] = 0.0
    far[:, 0] = -1024.0

    def spoil(d):
        v = d.pv[0][0] if prefix else d.v[0][s, 0]
        v[0, 7] = float("nan")
    nan = np.zeros((lay.tp, b.used, lay.hq, lay.d), bool)
    rows = slice(0, b.used) if prefix else slice(int(b.cu[s]), int(b.cu[s + 1]))
    nan[0, rows, :lay.group, 7] = True
    compare(b, run(gpu_lib, b, spoil), nan)


@pytest.mark.parametrize("form", list(FORMS))
def test_a_row_whose_scores_are_all_minus_infinity_is_nan(gpu_lib, form):
    # the weights' sum is 0 then, and 0 / 0 no number; zeros would pass for a result
    lay, new, cached, prefix = FORMS[form]
    b = K.Batch(lay, new, cached, prefix=prefix, seed=36)
    b.k[..., 0] = np.where(np.isnan(b.k[..., 0]), np.nan, -1.0)
    b.pk[..., 0] = -1.0
    t, r, h = b.used - 1, lay.tp - 1, lay.hq - 1

    def spoil(d):
        d.q[r, t, h, 0] = float("inf")
        d.q[0, 0, 0, 0] = float("inf")
    nan = np.zeros((lay.tp, b.used, lay.hq, lay.d), bool)
    nan[r, t, h] = nan[0, 0, 0] = True
    compare(b, run(gpu_lib, b, spoil), nan)


@pytest.mark.parametrize("form", ["whole_wide", "wide_parts", "narrow_parts", "few_rows", "few_rows_prefix", "shared_prefix"])
def test_keys_with_scores_of_minus_infinity_weigh_nothing(gpu_lib, form):
    # the first 256 keys of the longest cache, but not its last; the reference's have a score of -2^11 / sqrt(d), whose
    # weight is 0 beside the others' in every one of the bound's figures
    lay, new, cached, prefix = FORMS[form]
    b = K.Batch(lay, new, cached, prefix=prefix, seed=37)
    b.q[..., 0] = 1.0
    s = max(range(b.B), key=lambda i: cached[i])
    n = min(256, cached[s])
    b.k[0, s, 0, :n, 0] = -2048.0

    def spoil(d):
        d.k[0][s, 0, :n, 0] = -float("inf")
    compare(b, run(gpu_lib, b, spoil), np.zeros((lay.tp, b.used, lay.hq, lay.d), bool))
