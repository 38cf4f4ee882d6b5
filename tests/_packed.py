"""Packed batches for the tests: seeded inputs on the host, their attention in
float64, and the error that the kernels' roundings allow each element.

The bound, per output element with o = sum_j w_j v_j (sum_j w_j = 1) and
A = sum_j w_j |v_j|, both in float64:
  2^-8 |o|     the output's rounding to bf16 (half a step is 2^-8 relative),
  2^-8 A       each weight's rounding to bf16 (relative 2^-8 of every term),
  c A          float32 arithmetic: a score's d products and sums are off by at
               most (d + 2) 2^-24 sum|q_i k_i| / sqrt(d), which is the relative
               error of its weight and counts twice (numerator and normaliser);
               the exponential 2^-21; n additions n 2^-24, twice; the joining of
               parts and rescalings 2^-18,
with a factor 1 + 2^-6 on the sum for the products of these terms.
"""
import dataclasses

import numpy as np

import synth


def bf16(a):
    """float64 values after the rounding to bf16."""
    return synth.bf16_bits_as_f32(synth.round_to_bf16_bits(np.asarray(a, np.float32))).astype(np.float64)


@dataclasses.dataclass
class Layout:
    heads: int
    kv_heads: int
    d: int
    tp: int

    @property
    def hq(self):
        return self.heads // self.tp

    @property
    def hkv(self):
        return self.kv_heads // self.tp

    @property
    def group(self):
        return self.heads // self.kv_heads


class Batch:
    """Host inputs (float64 values that bf16 holds): q [tp, T, hq, d], caches [tp, B, hkv, max_kv, d]."""

    def __init__(self, lay: Layout, new, cached, prefix=0, extra_rows=0, extra_kv=0, seed=0, sharp=1.0, stale=np.nan,
                 max_kv=None):
        rng = np.random.default_rng(seed)
        self.lay, self.new, self.cached, self.prefix = lay, list(new), list(cached), prefix
        self.B = len(self.new)
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.used = int(self.cu[-1])
        self.T = max(1, self.used + extra_rows)
        self.max_kv = max_kv or max(1, max(n + c for n, c in zip(self.new, self.cached)) + extra_kv)
        self.q = bf16(sharp * rng.standard_normal((lay.tp, self.T, lay.hq, lay.d)))
        shape = (lay.tp, self.B, lay.hkv, self.max_kv, lay.d)
        self.k, self.v = bf16(rng.standard_normal(shape)), bf16(rng.standard_normal(shape))
        for b in range(self.B):                         # what an earlier sequence left behind the end
            end = min(self.new[b] + self.cached[b], self.max_kv)
            self.k[:, b, :, max(end, 0):] = stale
            self.v[:, b, :, max(end, 0):] = stale
        self.pk, self.pv = (bf16(rng.standard_normal((lay.tp, lay.hkv, prefix, lay.d))) for _ in range(2))

    def reference(self):
        """(o, bound) [tp, used, hq, d] in float64; rows outside the cache are zeros with bound 0."""
        lay, G = self.lay, self.lay.group
        o = np.zeros((lay.tp, self.used, lay.hq, lay.d))
        bound = np.zeros_like(o)
        for b in range(self.B):
            n, c = self.new[b], self.cached[b]
            if n == 0:
                continue
            end = max(min(n + c, self.max_kv), 0)
            keys = np.concatenate([self.pk, self.k[:, b, :, :end]], 2)
            vals = np.concatenate([self.pv, self.v[:, b, :, :end]], 2)
            pos = c + np.arange(n)
            live = (pos >= 0) & (pos < self.max_kv)
            hidden = np.arange(self.prefix + end)[None, :] > self.prefix + pos[:, None]
            for r in range(lay.tp):
                for h in range(lay.hq):
                    x = self.q[r, self.cu[b]:self.cu[b] + n, h]
                    K, V = keys[r, h // G], vals[r, h // G]
                    s = np.where(hidden, -np.inf, x @ np.nan_to_num(K).T / np.sqrt(lay.d))
                    s[~live] = 0.0
                    w = np.exp(s - s.max(-1, keepdims=True)) if s.size else s
                    w = w / w.sum(-1, keepdims=True)
                    mag = np.where(hidden, 0, np.abs(x) @ np.abs(np.nan_to_num(K)).T).max(-1, initial=0) / np.sqrt(lay.d)
                    nk = self.prefix + end
                    cc = 2 * (lay.d + 2) * 2.0 ** -24 * mag + 2.0 ** -21 + 2 * nk * 2.0 ** -24 + 2.0 ** -18
                    with np.errstate(invalid="ignore"):
                        seen = np.where(w[..., None] > 0, w[..., None] * V[None], 0.0) if not np.isfinite(V).all() else None
                        oo = w @ V if seen is None else seen.sum(1)
                        A = w @ np.abs(V) if seen is None else np.abs(seen).sum(1)
                    e = (1 + 2.0 ** -6) * (2.0 ** -8 * np.abs(oo) + (2.0 ** -8 + cc[:, None]) * A)
                    rows = slice(self.cu[b], self.cu[b] + n)
                    o[r, rows, h] = np.where(live[:, None], oo, 0)
                    bound[r, rows, h] = np.where(live[:, None], e, 0)
        return o, bound


def plan_desc(tb, lay: Layout, max_batch, max_tokens, max_kv, **kw):
    d = dict(hidden=64 * lay.heads, n_heads=lay.heads, n_kv_heads=lay.kv_heads, head_dim=lay.d, ffn=64 * lay.tp, n_experts=0,
             top_k=0, expert_ffn=0, org_vocab=0, eps=1e-5, rope_theta=5e5, dtype=tb.TP_BF16, has_qkv_bias=0,
             max_batch=max_batch, max_tokens=max_tokens, max_kv=max_kv, expert_parallel=0)
    return dict(d, **kw)


class OnDevice:
    """A batch's tensors, plan and workspace on the current device."""

    def __init__(self, tb, batch: Batch, prefix_extra=0, device="cuda"):
        import torch
        self.tb, self.b = tb, batch
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device).to(torch.bfloat16)  # noqa: E731
        self.q = dev(batch.q)
        self.k = [dev(a) for a in batch.k]
        self.v = [dev(a) for a in batch.v]
        self.prefix_rows = batch.prefix + prefix_extra
        pad = np.full((batch.lay.tp, batch.lay.hkv, prefix_extra, batch.lay.d), np.nan)
        self.pk = [dev(a) for a in np.concatenate([batch.pk, pad], 2)]
        self.pv = [dev(a) for a in np.concatenate([batch.pv, pad], 2)]
        self.cu = torch.from_numpy(batch.cu).to(device)
        self.pos = torch.tensor(batch.cached, dtype=torch.int32, device=device)
        self.out = torch.full_like(self.q, 7.0)
        self.plan = tb.tp_plan(plan_desc(tb, batch.lay, batch.B, batch.T, batch.max_kv), batch.lay.tp)
        self.nbytes = tb.tp_plan_get_info(self.plan)["workspace_bytes"]
        self.ws = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        tb.tp_workspace_init(self.plan, self.ws, self.nbytes)

    def run(self, stream=None):
        b = self.b
        if b.prefix:
            self.tb.tp_attn_prefix(self.plan, self.q, (self.pk, self.pv), b.prefix, self.prefix_rows, (self.k, self.v),
                                   self.cu, self.pos, b.B, b.T, self.out, self.ws, self.nbytes, stream)
        else:
            self.tb.tp_attn_packed(self.plan, self.q, (self.k, self.v), self.cu, self.pos, b.B, b.T, self.out, self.ws,
                                   self.nbytes, stream)
        return self.out

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
