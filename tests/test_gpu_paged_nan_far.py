"""NaN among the values of a prompt's last keys behind a long cache: the rows that
see it take it, the others are as without it, and the call ends in its time (the
waits of a kernel give up after a second)."""
import numpy as np
import pytest

from tests import _paged as K

pytestmark = pytest.mark.gpu

PAGE = 128


class Far:
    """`n` sequences of 40 new tokens behind `cached` keys, in pages that they share but for their last two."""

    def __init__(self, tb, lay, n, cached):
        import torch
        rng = np.random.default_rng(0)
        self.tb, self.lay, self.n, self.new, self.cached = tb, lay, n, 40, cached
        T = 40 * n
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16)  # noqa: E731
        self.q = dev(rng.standard_normal((lay.tp, T, lay.hq, lay.d)))
        self.out = torch.empty_like(self.q)
        need = -(-(cached + 40) // PAGE)
        table = rng.integers(0, 64, (n, need)).astype(np.int32)
        table[:, -2:] = 64 + np.arange(2 * n).reshape(n, 2)
        self.table = torch.from_numpy(table).cuda()
        shape = (64 + 2 * n, lay.hkv, PAGE, lay.d)
        self.pool = [torch.from_numpy(K.encode(64 * rng.standard_normal(shape))).cuda() for _ in range(2)]
        scale = torch.full(shape[:2], 2.0 ** -6, device="cuda")
        self.cu = torch.arange(0, T + 1, 40, dtype=torch.int32, device="cuda")
        self.pos = torch.full((n,), cached, dtype=torch.int32, device="cuda")
        self.plan = tb.tp_plan(K.plan_desc(tb, lay, n, T, 64), lay.tp)
        self.kv = tb.PagedKV(self.plan, [self.pool[0]], [self.pool[1]], [scale], [scale], self.table)
        self.bytes = tb.tp_paged_workspace_bytes(self.plan)
        self.ws = torch.empty(self.bytes, dtype=torch.uint8, device="cuda")
        tb.tp_paged_workspace_init(self.plan, self.ws, self.bytes)

    def attend(self):
        self.tb.tp_attn_paged(self.plan, self.q, self.kv, self.cu, self.pos, self.n, 40 * self.n, self.out, self.ws, self.bytes, 40)
        return self.out.float().cpu().numpy()


@pytest.mark.parametrize("lay,n,cached", [(K.Layout(32, 8, 128, 1), 19, 400000), (K.Layout(32, 8, 64, 1), 3, 30001),
                                          (K.Layout(4, 1, 128, 1), 1, 100)])
def test_nan_behind_a_long_cache(gpu_lib, lay, n, cached):
    f = Far(gpu_lib, lay, n, cached)
    spots = []                                  # (sequence, KV head, new token, feature)
    for s in range(n):
        for h in range(lay.hkv):
            i = (7 * s + 5 * h) % 40
            at = cached + i
            f.pool[1][int(f.table[s, at // PAGE]), h, at % PAGE, (11 * h + s) % lay.d] = 0x7F
            spots.append((s, h, i, (11 * h + s) % lay.d))
    got = f.attend()
    assert f.tb.tp_get_device_status(f.ws) == 0
    f.pool[1][f.pool[1] == 0x7F] = 0
    want = f.attend()
    assert np.isfinite(want).all()
    for s, h, i, x in spots:
        want[0, 40 * s + i:40 * s + 40, h * lay.group:(h + 1) * lay.group, x] = np.nan
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_blocks_that_lack_a_page(gpu_lib, d):
    """Pages outside the pool in the first and in a later block, with NaN in other pages of these and of whole blocks."""
    b = K.Batch(K.Layout(8, 2, d, 1), [40, 70], [1000, 300], 16)
    for s, w in ((0, 1), (0, 40), (1, 2)):
        b.table[s, w] = -1
    for s, p, x in ((0, 3, 1), (0, 200, 2), (0, 660, 3), (1, 50, 4), (1, 310, 5)):
        b.codes["v"][0, b.table[s, p // 16], 1, p % 16, x] = 0x7F
    dev = K.OnDevice(gpu_lib, b)
    dev.attend()
    assert gpu_lib.binding.STATUS_NAMES[dev.status()] == "TP_ERR_CAPACITY"
    got = np.isnan(dev.got())
    want = np.zeros_like(got)
    want[0, :40, 4:, 1:4] = True
    want[0, 40:, 4:, 4] = True
    want[0, 50:, 4:, 5] = True
    assert (got == want).all()
