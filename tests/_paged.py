"""8-bit paged caches for the tests: e4m3 in numpy, rotary embeddings, appending
and attention in float64, and the errors that the kernels' roundings allow.

Rotary embedding of a pair (a, b), by at most (|a| + |b|) m: the angle's fraction
of an eighth of a turn rounds by 2^-24 of pi / 4, sine and cosine are off by
2^-22, products and sum by 3 2^-24: together below 2^-21 (|a| + |b|) m; and the
frequency's fraction of a turn and its float64 logarithms by 2^-50 p f. A bf16
result adds 2^-8 of itself.

A stored value: half a step of its binade (2^-10 below 2^-6), and the rotation's
error over the scale. Scales, values without a rotation and values brought to a
larger scale have one right answer.

Attention, per element with o = sum_j w_j v_j and A = sum_j w_j |v_j|:
  2^-8 |o|     the output's rounding to bf16,
  2^-11 A      each weight's rounding to fp16, and its products with scales,
  n 2^-25 V    weights in fp16's subnormal range (V: the largest |v|), n keys,
  c A          a score of float32 products and sums, off by at most
               (2 d + 4) 2^-24 sum|q_i k_i| / sqrt(d) (the queries in two terms),
               and by 2^-17 max|q| sum|k_i| / sqrt(d) for queries held to 17 bits
               below a row's largest; its weight counts twice; the exponential
               2^-21; n additions n 2^-24, twice; joining and rescaling 2^-17,
with a factor 1 + 2^-6 on the sum for the products of these terms.
"""
import math

import numpy as np

from tests import _packed as K

bf16, Layout, plan_desc = K.bf16, K.Layout, K.plan_desc


def _table():
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.nan if c & 127 == 127 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        t[c] = -x if c & 128 else x
    return t


DECODE = _table()
_POSITIVE = DECODE[:127]                 # 0 .. 448, ascending


def encode(x):
    """e4m3 codes of values within +-448, to nearest even; what is not finite as NaN."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    up = a - _POSITIVE[lo] > _POSITIVE[hi] - a
    tie = a - _POSITIVE[lo] == _POSITIVE[hi] - a
    c = np.where(up | (tie & (hi % 2 == 0)), hi, lo)
    c = np.where(np.isfinite(x), c, 127) | np.where(np.signbit(x), 128, 0)
    return c.astype(np.uint8)


def half_step(x):
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    return 2.0 ** (e - 4)


def exponent(amax, growth):
    """The least e >= -60 with growth * amax <= 448 2^e."""
    need = np.asarray(amax, np.float64) * growth / 448
    e = np.full(need.shape, -60)
    big = need > 2.0 ** -60
    e[big] = np.ceil(np.log2(need[big])).astype(int)
    e[big] += 2.0 ** e[big] < need[big]
    e[big] -= 2.0 ** (e[big] - 1) >= need[big]
    return np.maximum(e, -60)


def rope_args(rot=0, layout=0, scaling=0, theta=0.0, factor=0.0, low=0.0, high=0.0, original=0, attn_factor=0.0):
    return dict(rot_dim=rot, layout=layout, scaling=scaling, theta=theta, factor=factor, low=low, high=high, original=original,
                attn_factor=attn_factor)


def frequencies(rope, d, plan_theta):
    """(f_i of every pair, m)."""
    rot, theta, s = rope["rot_dim"] or d, rope["theta"] or plan_theta, rope["factor"]
    f, m = [], rope["attn_factor"]
    for i in range(rot // 2):
        g = theta ** (-2 * i / rot)
        if rope["scaling"] == 1:
            g /= s
        elif rope["scaling"] == 2:
            turns = rope["original"] * g / (2 * math.pi)
            u = min(1.0, max(0.0, (turns - rope["low"]) / (rope["high"] - rope["low"])))
            g = (1 - u) * g / s + u * g
        elif rope["scaling"] == 3:
            c = lambda x: rot * math.log(rope["original"] / (2 * math.pi * x)) / (2 * math.log(theta))  # noqa: E731
            first, last = max(math.floor(c(rope["high"])), 0), min(math.ceil(c(rope["low"])), rot - 1)
            u = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            g = (1 - u) * g + u * g / s
        f.append(g)
    return np.array(f), m or (0.1 * math.log(s) + 1 if rope["scaling"] == 3 else 1.0)


def rotate(x, pos, rope, plan_theta):
    """([..., T, heads, d] turned, error bound) in float64."""
    d = x.shape[-1]
    rot = rope["rot_dim"] or d
    f, m = frequencies(rope, d, plan_theta)
    turns = np.array([[(int(p) * v / (2 * math.pi)) % 1.0 for v in f] for p in pos])
    angle = 2 * math.pi * turns[:, None, :]
    a = np.arange(rot // 2) if rope["layout"] == 0 else np.arange(0, rot, 2)
    b = a + (rot // 2 if rope["layout"] == 0 else 1)
    y, e = np.array(x), np.zeros_like(x)
    with np.errstate(invalid="ignore"):
        y[..., a] = m * (x[..., a] * np.cos(angle) - x[..., b] * np.sin(angle))
        y[..., b] = m * (x[..., a] * np.sin(angle) + x[..., b] * np.cos(angle))
        far = np.abs(np.array([int(p) for p in pos], np.float64))[:, None, None] * f * 2.0 ** -50
        e[..., a] = e[..., b] = m * (np.abs(x[..., a]) + np.abs(x[..., b])) * (2.0 ** -21 + far)
    return y, e


class Batch:
    """Host inputs of a packed batch over pages: stored codes [tp][pages][hkv][page][d] and scales, a table of shuffled pages
    with -1 behind a sequence's last; free slots hold NaN. Exponents of the scales spread by `spread`."""

    def __init__(self, lay: Layout, new, cached, page=16, extra_rows=0, extra_pages=0, seed=0, sharp=1.0, spread=3, width=None,
                 stale=0x7F):
        rng = np.random.default_rng(seed)
        self.lay, self.new, self.cached, self.page, self.rng = lay, list(new), list(cached), page, rng
        self.B = len(self.new)
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.used = int(self.cu[-1])
        self.T = max(1, self.used + extra_rows)
        self.q = bf16(sharp * rng.standard_normal((lay.tp, self.T, lay.hq, lay.d)))
        self.new_k = bf16(rng.standard_normal((lay.tp, self.T, lay.hkv, lay.d)))
        self.new_v = bf16(rng.standard_normal((lay.tp, self.T, lay.hkv, lay.d)))
        need = [max(0, -(-(n + c) // page)) for n, c in zip(self.new, self.cached)]
        self.width = width or max(1, max(need) + extra_pages)
        self.n_pages = sum(need) + 2
        order = rng.permutation(self.n_pages)
        self.table = np.full((self.B, self.width), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            m = min(m, self.width)
            self.table[b, :m] = order[at:at + m]
            at += m
        shape = (lay.tp, self.n_pages, lay.hkv, page, lay.d)
        self.scale, self.codes = {}, {}
        for name in "kv":
            x = rng.standard_normal(shape) * 2.0 ** rng.integers(-spread, spread + 1, shape[:3])[..., None, None]
            e = exponent(np.abs(x).max((3, 4)), 1.0)
            self.scale[name] = 2.0 ** e
            self.codes[name] = encode(x / self.scale[name][..., None, None])
            free = np.ones(shape[:2] + (page,), bool)
            for b in range(self.B):
                for j in range(min(max(self.new[b] + self.cached[b], 0), self.width * page)):
                    free[:, self.table[b, j // page], j % page] = False
            self.codes[name][np.broadcast_to(free[:, :, None, :], shape[:4])] = stale

    def keys(self, name, b, r, n):
        """float64 [hkv][n][d] of a sequence's first n slots."""
        ids = self.table[b, :-(-n // self.page)]
        x = DECODE[self.codes[name][r, ids]] * self.scale[name][r, ids][..., None, None]
        return x.transpose(1, 0, 2, 3).reshape(self.lay.hkv, -1, self.lay.d)[:, :n]

    def positions(self):
        return np.concatenate([c + np.arange(n) for n, c in zip(self.new, self.cached)] + [np.zeros(0, int)]).astype(np.int64)

    def reference(self):
        """Attention: (o, bound) [tp, used, hq, d]; rows outside the pages are zeros with bound 0."""
        lay, G, cap = self.lay, self.lay.group, self.width * self.page
        o = np.zeros((lay.tp, self.used, lay.hq, lay.d))
        bound = np.zeros_like(o)
        for b in range(self.B):
            n, c = self.new[b], self.cached[b]
            end = max(min(n + c, cap), 0)
            pos = c + np.arange(n)
            live = (pos >= 0) & (pos < cap)
            if not live.any():
                continue
            hidden = np.arange(end)[None, :] > pos[:, None]
            for r in range(lay.tp):
                keys, vals = self.keys("k", b, r, end), self.keys("v", b, r, end)
                for h in range(lay.hq):
                    x = self.q[r, self.cu[b]:self.cu[b] + n, h]
                    k, v = keys[h // G], vals[h // G]
                    s = np.where(hidden, -np.inf, x @ k.T / np.sqrt(lay.d))
                    s[~live] = 0.0
                    w = np.exp(s - s.max(-1, keepdims=True))
                    w = w / w.sum(-1, keepdims=True)
                    mag = np.where(hidden, 0, np.abs(x) @ np.abs(k).T).max(-1) / np.sqrt(lay.d)
                    low = 2.0 ** -17 * np.abs(x).max(-1) * np.abs(k).sum(-1).max() / np.sqrt(lay.d)
                    cc = 2 * (2 * lay.d + 4) * 2.0 ** -24 * mag + 2 * low + 2.0 ** -21 + 2 * end * 2.0 ** -24 + 2.0 ** -17
                    oo, A = w @ v, w @ np.abs(v)
                    e = (1 + 2.0 ** -6) * (2.0 ** -8 * np.abs(oo) + (2.0 ** -11 + cc[:, None]) * A +
                                           end * 2.0 ** -25 * np.abs(v).max())
                    rows = slice(self.cu[b], self.cu[b] + n)
                    o[r, rows, h] = np.where(live[:, None], oo, 0)
                    bound[r, rows, h] = np.where(live[:, None], e, 0)
        return o, bound

    def appended(self, rope, plan_theta):
        """What tp_kv_append_paged leaves: {name: (codes, bound in steps of the stored values or None, scales)}, of which a
        bound of 0 means that the code is the right one."""
        lay, page, cap = self.lay, self.page, self.width * self.page
        pos = self.positions()
        out = {}
        m = frequencies(rope, lay.d, plan_theta)[1] if rope else 1.0
        for name, given in (("k", self.new_k[:, :self.used]), ("v", self.new_v[:, :self.used])):
            turned, err = rotate(given, pos, rope, plan_theta) if rope and name == "k" else (given, np.zeros_like(given))
            growth = math.sqrt(2.0) * max(1.0, m) if rope and name == "k" else 1.0
            codes, scale = self.codes[name].copy(), self.scale[name].copy()
            value, bound = DECODE[codes], np.zeros(codes.shape)
            for b in range(self.B):
                for w in range(self.cached[b] // page, -(-(self.cached[b] + self.new[b]) // page)):
                    lo, hi = max(w * page, self.cached[b]), min((w + 1) * page, self.cached[b] + self.new[b])
                    if lo >= hi or lo < 0 or lo >= cap:
                        continue
                    at, rows = self.table[b, w], slice(self.cu[b] + lo - self.cached[b], self.cu[b] + hi - self.cached[b])
                    if at < 0 or at >= self.n_pages:
                        continue
                    x = given[:, rows]
                    s = 2.0 ** exponent(np.where(np.isfinite(x), np.abs(x), 0).max((1, 3)), growth)
                    if lo > w * page:
                        s = np.maximum(s, scale[:, at])
                        kept = DECODE[codes[:, at]] * (scale[:, at] / s)[..., None, None]
                        codes[:, at] = encode(kept)
                        value[:, at] = DECODE[codes[:, at]]
                    scale[:, at] = s
                    slots = slice(lo - w * page, hi - w * page)
                    y = turned[:, rows].transpose(0, 2, 1, 3) / s[..., None, None]
                    e = err[:, rows].transpose(0, 2, 1, 3) / s[..., None, None]
                    codes[:, at, :, slots] = encode(y)
                    value[:, at, :, slots] = y
                    with np.errstate(invalid="ignore"):
                        bound[:, at, :, slots] = np.where((e > 0) & np.isfinite(y), half_step(y) + e, 0)
            out[name] = (codes, value, bound, scale)
        return out


class OnDevice:
    """A batch's tensors, plan and workspace on the current device."""

    def __init__(self, tb, batch: Batch, max_new=0, device="cuda", theta=5e5):
        import torch
        self.tb, self.b, self.max_new = tb, batch, max_new
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device).to(torch.bfloat16)  # noqa: E731
        self.q, self.new_k, self.new_v = dev(batch.q), dev(batch.new_k), dev(batch.new_v)
        self.pool = {n: [torch.from_numpy(a.copy()).to(device) for a in batch.codes[n]] for n in "kv"}
        self.scale = {n: [torch.from_numpy(a.astype(np.float32)).to(device) for a in batch.scale[n]] for n in "kv"}
        self.table = torch.from_numpy(batch.table).to(device)
        self.cu = torch.from_numpy(batch.cu).to(device)
        self.pos = torch.tensor(batch.cached, dtype=torch.int32, device=device)
        self.out = torch.full_like(self.q, 7.0)
        self.plan = tb.tp_plan(plan_desc(tb, batch.lay, batch.B, batch.T, 64, rope_theta=theta), batch.lay.tp)
        self.kv = tb.PagedKV(self.plan, self.pool["k"], self.pool["v"], self.scale["k"], self.scale["v"], self.table)
        self.nbytes = tb.tp_paged_workspace_bytes(self.plan)
        self.ws = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        tb.tp_paged_workspace_init(self.plan, self.ws, self.nbytes)
        self.word = torch.zeros(1, dtype=torch.int32, device=device)

    def attend(self, stream=None):
        self.tb.tp_attn_paged(self.plan, self.q, self.kv, self.cu, self.pos, self.b.B, self.b.T, self.out, self.ws, self.nbytes,
                              self.max_new, stream)
        return self.out

    def append(self, rope=None, q=None, q_out=None, stream=None):
        self.tb.tp_kv_append_paged(self.plan, self.tb.tp_rope(**rope) if rope else None, self.new_k, self.new_v, self.kv, self.cu,
                                   self.pos, self.b.B, self.b.T, q=q, q_out=q_out, device_status=self.word, stream=stream)

    def status(self):
        return self.tb.tp_get_device_status(self.ws)

    def got(self):
        return self.out.double().cpu().numpy()


def check(got, batch: Batch, ref=None):
    """Rows in use within the bound, rows behind them untouched; returns the largest share of the bound."""
    o, bound = ref or batch.reference()
    g = got[:, :batch.used]
    assert np.isfinite(g).all()
    diff = np.abs(g - o)
    assert (diff <= bound).all(), (float((diff - bound).max()), np.argwhere(diff > bound)[:5].tolist())
    assert (got[:, batch.used:] == 7.0).all()
    return float((diff / np.maximum(bound, 1e-30)).max()) if diff.size else 0.0
