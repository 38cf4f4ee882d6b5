"""Lists of the logit controls whose offsets do not lie in them: such a row has
an empty list, and the others keep theirs."""
import numpy as np
import pytest

from tests.test_gpu_logits import Case, plan_of

pytestmark = pytest.mark.gpu

# offsets of four rows into a list of 20 entries, and rows that have the list of 5 entries that they would have otherwise
OFFSETS = {
    "end_behind": ([0, 5, 10, 15, 21], [0, 1, 2]),
    "far_behind": ([0, 5, 10, 2 ** 31 - 1, 20], [0, 1]),
    "begin_below": ([-1, 5, 10, 15, 20], [1, 2, 3]),
    "far_below": ([0, -2 ** 31, 10, 15, 20], [2, 3]),
    "decreasing": ([0, 5, 4, 15, 20], [0, 3]),
    "all_behind": ([2 ** 30, 2 ** 30 + 5, 2 ** 30 + 10, 2 ** 30 + 15, 2 ** 30 + 20], []),
    "exactly": ([0, 5, 10, 15, 20], [0, 1, 2, 3]),
}


@pytest.mark.parametrize("which", ["tokens", "bias", "both"])
@pytest.mark.parametrize("name", list(OFFSETS))
def test_offsets_outside_a_list_give_an_empty_one(gpu_lib, name, which):
    import torch
    cu, keep = OFFSETS[name]
    c = Case(T=4, V=9001, seed=71, masks=4)
    rng = np.random.default_rng(72)
    c.hist = [rng.integers(0, 9001, 5).tolist() for _ in range(4)]
    c.n_prompt = np.array([2, 0, 5, 1], np.int32)
    c.bias = [[(int(v), float(np.float32(z))) for v, z in zip(rng.integers(0, 9001, 5), rng.standard_normal(5))] for _ in range(4)]
    kw = c.args(torch)
    bad = torch.tensor(cu, dtype=torch.int64).to(torch.int32).cuda()
    spans = {t: (cu[t], cu[t + 1]) for t in range(4) if 0 <= cu[t] < cu[t + 1] <= 20}
    if which in ("tokens", "both"):
        flat = [v for h in c.hist for v in h]
        kw["cu_tokens"] = bad
        c.hist = [flat[slice(*spans[t])] if t in spans else [] for t in range(4)]
    if which in ("bias", "both"):
        flat = [x for b in c.bias for x in b]
        kw["cu_bias"] = bad
        c.bias = [flat[slice(*spans[t])] if t in spans else [] for t in range(4)]
    assert set(keep) <= set(spans)
    out = torch.empty(4, 9001, device="cuda")
    gpu_lib.tp_logits_process(plan_of(gpu_lib, 9001), torch.from_numpy(c.x).cuda(), 4, out, **kw)
    c.check(out.cpu().numpy())


def test_a_shorter_length_than_the_tensor_holds(gpu_lib):
    import torch
    c = Case(T=2, V=500, seed=73, max_bias=None)
    c.hist = [[1, 2, 3], [4, 4, 5]]
    c.n_prompt = np.array([1, 0], np.int32)
    kw = c.args(torch)
    c.hist[1] = []                               # its last entry lies behind the length given
    out = torch.empty(2, 500, device="cuda")
    gpu_lib.tp_logits_process(plan_of(gpu_lib, 500), torch.from_numpy(c.x).cuda(), 2, out, n_tokens=5, **kw)
    c.check(out.cpu().numpy())


def test_fewer_values_than_biased_tokens_are_refused(gpu_lib):
    import torch
    c = Case(T=2, V=500, seed=74, max_bias=9)
    kw = c.args(torch)
    kw["bias_values"] = kw["bias_values"][:-1].clone()
    x = torch.from_numpy(c.x).cuda()
    with pytest.raises(ValueError, match="bias_values"):
        gpu_lib.tp_logits_process(plan_of(gpu_lib, 500), x, 2, torch.empty_like(x), **kw)


@pytest.mark.parametrize("which", ["tokens", "bias", "both"])
def test_a_batch_without_any_entries(gpu_lib, which):
    # the first step of requests without a history: empty tensors, whose address is NULL
    import torch
    c = Case(T=3, V=700, seed=75, masks=3)
    if which in ("tokens", "both"):
        c.hist = [[], [], []]
        c.n_prompt = np.zeros(3, np.int32)
    if which in ("bias", "both"):
        c.bias = [[], [], []]
    kw = c.args(torch)
    if which in ("tokens", "both"):
        kw["tokens"] = torch.empty(0, dtype=torch.int32, device="cuda")
    if which in ("bias", "both"):
        kw["bias_ids"] = torch.empty(0, dtype=torch.int32, device="cuda")
        kw["bias_values"] = torch.empty(0, device="cuda")
    if which == "both":                          # nor a row with a grammar
        kw["mask"] = torch.empty(0, 22, dtype=torch.int32, device="cuda")
        kw["mask_row"] = torch.full((3,), -1, dtype=torch.int32, device="cuda")
        c.mask = None
    x = torch.from_numpy(c.x).cuda()
    out = torch.empty_like(x)
    gpu_lib.tp_logits_process(plan_of(gpu_lib, 700), x, 3, out, **kw)
    c.check(out.cpu().numpy())
    with pytest.raises(TypeError):               # what goes with an empty list is checked all the same
        gpu_lib.tp_logits_process(plan_of(gpu_lib, 700), x, 3, out, **{**kw, "repetition": kw["repetition"].double()})
