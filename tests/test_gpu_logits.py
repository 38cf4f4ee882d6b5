"""Per-row controls of logits against float64. Each of the at most five
float32 operations on a logit (division or product, product, two subtractions,
addition) is off by at most 2^-24 of its result's size, so an entry's error is
at most 5 * 2^-24 times the largest intermediate size, taken as
|x| max(r, 1/r) + |f| c + |a| + |bias|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def reference(x, hist, n_prompt, rep, pres, freq, bias, mask, mask_row):
    y = x.astype(np.float64).copy()
    size = np.abs(y)
    T, V = x.shape
    for t in range(T):
        h = [v for v in hist[t]]
        gen = {}
        for v in h[n_prompt[t] if n_prompt is not None else 0:]:
            if 0 <= v < V:
                gen[v] = gen.get(v, 0) + 1
        r, a, f = (float(p[t]) if p is not None else n for p, n in ((rep, 1.0), (pres, 0.0), (freq, 0.0)))
        for v in {v for v in h if 0 <= v < V}:
            y[t, v] = y[t, v] / r if y[t, v] > 0 else y[t, v] * r
            size[t, v] *= max(r, 1 / r)
        for v, c in gen.items():
            y[t, v] = y[t, v] - f * c - a
            size[t, v] += abs(f) * c + abs(a)
        if bias is not None:
            for v, z in dict(bias[t]).items():          # the last of a token's entries
                if 0 <= v < V:
                    y[t, v] += z
                    size[t, v] += abs(z)
        if mask is not None:
            m = mask_row[t] if mask_row is not None else t
            if 0 <= m < mask.shape[0]:
                bits = ((mask[m][:, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(-1)[:V]
                y[t, bits == 0] = -np.inf
    return y, 5 * 2.0 ** -24 * size


class Case:
    def __init__(self, T, V, seed, max_hist=50, max_bias=8, masks=None, penalties=True, prompt=True, wild=False):
        rng = np.random.default_rng(seed)
        self.T, self.V = T, V
        self.x = (3 * rng.standard_normal((T, V))).astype(np.float32)
        pick = (lambda n: rng.integers(-3, V + 3, n)) if wild else (lambda n: (V * rng.random(n) ** 3).astype(int))
        self.hist = [pick(rng.integers(0, max_hist + 1)).tolist() for _ in range(T)]
        self.n_prompt = np.array([rng.integers(0, len(h) + 2) for h in self.hist], np.int32) if prompt else None
        self.rep, self.pres, self.freq = ((1 + rng.random(T)).astype(np.float32), rng.standard_normal(T).astype(np.float32),
                                          rng.standard_normal(T).astype(np.float32)) if penalties else (None,) * 3
        self.bias = None
        if max_bias is not None:
            self.bias = []
            for _ in range(T):
                ids = pick(rng.integers(0, max_bias + 1)).tolist()
                self.bias.append(list(zip(ids, (10 * rng.standard_normal(len(ids))).astype(np.float32).tolist())))
        self.mask = self.mask_row = None
        if masks is not None:
            self.mask = rng.integers(0, 1 << 32, (masks, (V + 31) // 32), dtype=np.uint64).astype(np.uint32)
            if masks != T:
                self.mask_row = rng.integers(-1, masks, T).astype(np.int32)

    def args(self, torch):
        i32 = lambda a: torch.tensor(np.asarray(a, np.int64), device="cuda").to(torch.int32)  # noqa: E731
        f32 = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.float32)).to("cuda")  # noqa: E731
        flat = lambda ls: [v for l in ls for v in l]  # noqa: E731
        cum = lambda ls: i32(np.concatenate([[0], np.cumsum([len(l) for l in ls])]))  # noqa: E731
        kw = dict(tokens=i32(flat(self.hist)), cu_tokens=cum(self.hist), repetition=f32(self.rep), presence=f32(self.pres),
                  frequency=f32(self.freq), n_prompt=None if self.n_prompt is None else i32(self.n_prompt))
        if not flat(self.hist):
            kw["tokens"] = i32([0])
        if self.bias is not None:
            b = flat(self.bias)
            kw.update(bias_ids=i32([v for v, _ in b] or [0]), bias_values=f32([z for _, z in b] or [0.0]),
                      cu_bias=cum(self.bias))
        if self.mask is not None:
            kw.update(mask=torch.from_numpy(self.mask.view(np.int32)).to("cuda"))
            if self.mask_row is not None:
                kw.update(mask_row=i32(self.mask_row))
        return kw

    def check(self, got):
        y, e = reference(self.x, self.hist, self.n_prompt, self.rep, self.pres, self.freq, self.bias, self.mask,
                         self.mask_row)
        fine = np.isfinite(y)
        assert np.array_equal(got[~fine], y[~fine])
        d = np.abs(got.astype(np.float64) - y)
        assert (d[fine] <= e[fine]).all(), float((d - e)[fine].max())


def plan_of(tb, V):
    return tb.tp_plan(dict(hidden=64, n_heads=1, n_kv_heads=1, head_dim=64, ffn=64, n_experts=0, top_k=0, expert_ffn=0,
                           org_vocab=V, eps=1e-5, rope_theta=5e5, dtype=tb.TP_BF16, has_qkv_bias=0, max_batch=1,
                           max_tokens=1, max_kv=1, expert_parallel=0), 1)


CASES = {
    "one_row_1000": dict(T=1, V=1000, masks=1),
    "vocab_1": dict(T=3, V=1, masks=3, max_hist=4),
    "vocab_2_to_rows": dict(T=7, V=2, masks=2),
    "vocab_33_odd_rows": dict(T=5, V=33, masks=5),
    "vocab_8191": dict(T=3, V=8191, masks=2, max_hist=3000),
    "vocab_8193": dict(T=4, V=8193, masks=4, max_hist=3000),
    "vocab_50257": dict(T=9, V=50257, masks=3, max_hist=2000, max_bias=300),
    "vocab_151936": dict(T=8, V=151936, masks=8, max_hist=4000, max_bias=300),
    "many_rows": dict(T=300, V=777, masks=100),
    "ids_outside": dict(T=6, V=100, masks=6, wild=True),
    "only_masks": dict(T=6, V=5000, masks=3, max_hist=0, max_bias=None, penalties=False),
    "only_penalties": dict(T=6, V=5001, max_bias=None),
    "only_biases": dict(T=6, V=5002, max_hist=0, max_bias=700, penalties=False),
    "no_prompt_counts": dict(T=6, V=300, prompt=False, max_hist=900),
    "one_token_again_and_again": dict(T=2, V=3, max_hist=70000, masks=None),
    "full_bias": dict(T=2, V=600, max_bias=5000),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_controls_match_float64(gpu_lib, name, in_place):
    import torch
    c = Case(seed=len(name), **CASES[name])
    plan = plan_of(gpu_lib, c.V)
    x = torch.from_numpy(c.x).to("cuda")
    guard = torch.full((c.T * c.V + 64,), 7.0, device="cuda")
    out = x if in_place else guard[:c.T * c.V].view(c.T, c.V)
    gpu_lib.tp_logits_process(plan, x, c.T, out, **c.args(torch))
    c.check(out.cpu().numpy())
    assert (guard[c.T * c.V:] == 7.0).all()
    if not in_place:
        assert np.array_equal(x.cpu().numpy(), c.x)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_buffers_off_16_bytes(gpu_lib, shift):
    import torch
    c = Case(T=5, V=10001, seed=3, masks=5, max_hist=500)
    plan = plan_of(gpu_lib, c.V)
    n = c.T * c.V
    x = torch.zeros(n + 8, device="cuda")[shift:shift + n].view(c.T, c.V)
    x.copy_(torch.from_numpy(c.x))
    out = torch.full((n + 8,), 7.0, device="cuda")
    gpu_lib.tp_logits_process(plan, x, c.T, out[shift:shift + n].view(c.T, c.V), **c.args(torch))
    got = out.cpu().numpy()
    c.check(got[shift:shift + n].reshape(c.T, c.V))
    assert (got[:shift] == 7).all() and (got[shift + n:] == 7).all()


def test_no_controls_copies_and_leaves_in_place(gpu_lib):
    import torch
    x = torch.randn(3, 999, device="cuda")
    plan = plan_of(gpu_lib, 999)
    out = torch.empty_like(x)
    gpu_lib.tp_logits_process(plan, x, 3, out)
    assert torch.equal(out, x)
    before = x.clone()
    gpu_lib.tp_logits_process(plan, x, 3, x)
    assert torch.equal(before, x)


def test_infinities_and_nan_in_logits(gpu_lib):
    import torch
    c = Case(T=4, V=500, seed=9, masks=4)
    plan = plan_of(gpu_lib, c.V)
    x = torch.from_numpy(c.x).to("cuda")
    x[0, 3], x[1, 4], x[2, 5], x[3, 6] = float("nan"), float("inf"), float("-inf"), float("nan")
    out = torch.empty_like(x)
    gpu_lib.tp_logits_process(plan, x, c.T, out, **c.args(torch))
    bits = lambda t, v: (int(c.mask[t, v // 32]) >> (v % 32)) & 1  # noqa: E731
    for t, v, want in ((0, 3, float("nan")), (1, 4, float("inf")), (2, 5, float("-inf")), (3, 6, float("nan"))):
        got = out[t, v].item()
        want = want if bits(t, v) else float("-inf")
        assert (got != got) if want != want else got == want
    y = out.clone()
    y[0, 3] = y[1, 4] = y[2, 5] = y[3, 6] = 0.0
    c.x[0, 3] = c.x[1, 4] = c.x[2, 5] = c.x[3, 6] = 0.0
    z = torch.empty_like(x)
    gpu_lib.tp_logits_process(plan, torch.from_numpy(c.x).to("cuda"), c.T, z, **c.args(torch))
    z[0, 3] = z[1, 4] = z[2, 5] = z[3, 6] = 0.0
    assert torch.equal(y, z)


def test_captured_and_on_another_stream(gpu_lib):
    import torch
    c = Case(T=8, V=20000, seed=5, masks=8, max_hist=800)
    plan, kw = plan_of(gpu_lib, c.V), c.args(torch)
    x = torch.from_numpy(c.x).to("cuda")
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gpu_lib.tp_logits_process(plan, x, c.T, out, stream=s, **kw)
    s.synchronize()
    c.check(out.cpu().numpy())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.tp_logits_process(plan, x, c.T, out, **kw)
    other = Case(T=8, V=20000, seed=6, masks=8, max_hist=800)
    x.copy_(torch.from_numpy(other.x))
    other.hist, other.n_prompt, other.rep, other.pres, other.freq = c.hist, c.n_prompt, c.rep, c.pres, c.freq
    other.bias, other.mask, other.mask_row = c.bias, c.mask, c.mask_row
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    other.check(out.cpu().numpy())
