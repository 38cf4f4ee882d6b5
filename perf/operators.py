"""Cases, plain forms and 64-bit values of three serving operators of the
tensor-parallel block library: attention of a packed batch of prompts over the
sharded KV caches (``tp_attn_packed``), the same for a batch whose sequences
share a long prefix (``tp_attn_prefix``), and the per-request controls of a
batch's logits (``tp_logits_process``).

Head layouts, shard counts and the vocabulary are those of the workloads in
``synth.py``; the others are generic.
"""
import math
import random

import torch

own = False

# (query heads, KV heads, head size, shards): the Llama-3-8B-shaped and Qwen2.5-0.5B-shaped layers of synth.py
LLAMA_TP8 = dict(heads=32, kv_heads=8, head_dim=128, tp=8)
LLAMA_TP4 = dict(heads=32, kv_heads=8, head_dim=128, tp=4)
QWEN_TP2 = dict(heads=14, kv_heads=2, head_dim=64, tp=2)
VOCAB = 151936

PROMPT_KEYS = ("batch", "min_new", "max_new", "min_cached", "max_cached", "lens_seed")


def _prompt(name, layout, batch, min_new, max_new, min_cached, max_cached, lens_seed, prefix=None):
    c = {"name": name, "op": "packed" if prefix is None else "prefix", **layout, "batch": batch, "min_new": min_new,
         "max_new": max_new, "min_cached": min_cached, "max_cached": max_cached, "lens_seed": lens_seed}
    if prefix is not None:
        c["prefix"] = prefix
    return c


def listed():
    return [
        # one new token of one sequence over a cache of 512: the smallest call, all latency
        _prompt("packed_one_token", QWEN_TP2, 1, 1, 1, 512, 512, 1),
        # many short requests of a busy server, some continuing a cached conversation
        _prompt("packed_short_requests", QWEN_TP2, 64, 1, 512, 0, 512, 2),
        # a prefill batch of unlike prompts, none cached
        _prompt("packed_ragged_prompts", LLAMA_TP8, 12, 1, 2048, 0, 0, 3),
        # one chunk of a long prompt that is prefilled piece by piece
        _prompt("packed_chunk_of_long", LLAMA_TP4, 1, 512, 512, 30001, 30001, 4),
        # one long document
        _prompt("packed_long_prompt", LLAMA_TP8, 1, 16384, 16384, 0, 0, 5),
        # a few chats behind one short system prompt, one token each: latency
        _prompt("prefix_small_batch", QWEN_TP2, 4, 1, 1, 0, 63, 6, prefix=777),
        # a decode step of 64 chats behind a long system prompt
        _prompt("prefix_decode_64", LLAMA_TP4, 64, 1, 1, 0, 1023, 7, prefix=4096),
        # a decode step of many requests over one long shared document
        _prompt("prefix_decode_256", LLAMA_TP4, 256, 1, 1, 0, 2047, 8, prefix=16384),
        # questions of unlike lengths on one shared text, prefilled together
        _prompt("prefix_questions", LLAMA_TP8, 16, 1, 512, 0, 0, 9, prefix=2048),
        # one request's logits: a history to penalise, a few biases
        {"name": "logits_one_row", "op": "logits", "rows": 1, "vocab": VOCAB, "max_history": 700, "max_bias": 16,
         "masks": 0, "lens_seed": 10},
        # a decode batch of eight, half of them held to a grammar
        {"name": "logits_batch_8", "op": "logits", "rows": 8, "vocab": VOCAB, "max_history": 4096, "max_bias": 300,
         "masks": 4, "lens_seed": 11},
        # a large batch with long histories, every row with a grammar of its own
        {"name": "logits_batch_256", "op": "logits", "rows": 256, "vocab": VOCAB, "max_history": 8192, "max_bias": 100,
         "masks": 256, "lens_seed": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["packed", "packed", "prefix", "prefix", "logits"])
    if op == "logits":
        rows = _log_int(rng, 1, 256)
        return {"op": op, "rows": rows, "vocab": rng.choice([VOCAB, _log_int(rng, 1000, VOCAB)]),
                "max_history": _log_int(rng, 1, 8192), "max_bias": rng.choice([0, _log_int(rng, 1, 300)]),
                "masks": rng.choice([0, rng.randint(1, rows)]), "lens_seed": rng.randint(100, 1 << 30)}
    while True:
        group, kv = rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), rng.choice([1, 2, 4, 8])
        layout = rng.choice([QWEN_TP2, LLAMA_TP4, LLAMA_TP8,
                             dict(heads=group * kv, kv_heads=kv, head_dim=rng.choice([64, 128]),
                                  tp=rng.choice([t for t in (1, 2, 4, 8) if kv % t == 0]))])
        if op == "packed":
            batch, most = _log_int(rng, 1, 128), _log_int(rng, 1, 8192)
        else:
            batch, most = _log_int(rng, 1, 256), rng.choice([1, 1, _log_int(rng, 1, 1024)])
        cached = rng.choice([0, _log_int(rng, 1, 16384 if op == "packed" else 2047)])
        c = {"op": op, **layout, "batch": batch, "min_new": 1 if batch > 1 else max(1, most // 2), "max_new": most,
             "min_cached": 0, "max_cached": cached, "lens_seed": rng.randint(100, 1 << 30)}
        if op == "prefix":
            c["prefix"] = _log_int(rng, 1, 16384)
        # the plain form pads every sequence to the longest: keep its scores, and its copies of the keys, of a size it can hold
        w = work(c)
        scores = batch * c["heads"] * most * (most + cached + c.get("prefix", 0))
        keys = batch * c["kv_heads"] * (most + cached) * c["head_dim"]
        if w["flops"] <= 2e12 and w["bytes"] <= 1.2e9 and scores <= 4e9 and keys <= 1.2e9:
            return c


def _lens(case):
    """Lengths of a batch, from the case alone: (new tokens, cached tokens) of every sequence."""
    rng = random.Random(case["lens_seed"])
    new = [_log_int(rng, case["min_new"], case["max_new"]) for _ in range(case["batch"])]
    cached = [rng.randint(case["min_cached"], case["max_cached"]) for _ in range(case["batch"])]
    return new, cached


def _logit_lens(case):
    rng = random.Random(case["lens_seed"])
    history = [rng.randint(0, case["max_history"]) if case["rows"] > 1 else case["max_history"] for _ in range(case["rows"])]
    prompt = [rng.randint(0, h) for h in history]
    bias = [rng.randint(0, case["max_bias"]) for _ in range(case["rows"])]
    mask_row = list(range(case["masks"])) + [-1] * (case["rows"] - case["masks"])
    rng.shuffle(mask_row)
    return history, prompt, bias, mask_row


def work(case):
    if case["op"] == "logits":
        history, _, bias, _ = _logit_lens(case)
        cells = case["rows"] * case["vocab"]
        return {"bytes": 8 * cells + case["masks"] * ((case["vocab"] + 31) // 32) * 4 + 4 * sum(history) + 8 * sum(bias),
                "flops": cells + 4 * sum(history) + sum(bias)}
    new, cached = _lens(case)
    d, heads, kv_heads, prefix = case["head_dim"], case["heads"], case["kv_heads"], case.get("prefix", 0)
    tokens = sum(new)
    seen = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, cached)) + tokens * prefix
    keys = sum(n + c for n, c in zip(new, cached)) + prefix
    return {"bytes": 2 * (2 * tokens * heads * d + 2 * keys * kv_heads * d), "flops": 4 * d * heads * seen}


def _cumulative(lens, device):
    return torch.tensor([0] + lens, device=device).cumsum(0).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    return (_prepare_logits if case["op"] == "logits" else _prepare_attention)(case, g, dev)


def _prepare_attention(case, g, dev):
    new, cached = _lens(case)
    n, heads, kv, d = case["tp"], case["heads"] // case["tp"], case["kv_heads"] // case["tp"], case["head_dim"]
    tokens, rows = sum(new), max(a + b for a, b in zip(new, cached))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    s = {"case": case, "tokens": tokens, "longest": max(new), "rows": rows}
    # queries of some heads are sharper than others', as in a trained layer
    sharp = 0.5 + 2.5 * torch.rand(n, 1, heads, 1, generator=g, device=dev)
    s["q"] = (normal(n, tokens, heads, d) * sharp).to(torch.bfloat16)
    # per shard the cache of every sequence [batch][KV heads][rows][d]; rows past a sequence's end hold what an earlier one left
    s["k"] = [normal(case["batch"], kv, rows, d) for _ in range(n)]
    s["v"] = [normal(case["batch"], kv, rows, d) for _ in range(n)]
    s["cu"], s["pos"] = _cumulative(new, dev), torch.tensor(cached, device=dev, dtype=torch.int32)
    if case["op"] == "prefix":
        s["pk"] = [normal(kv, case["prefix"], d) for _ in range(n)]
        s["pv"] = [normal(kv, case["prefix"], d) for _ in range(n)]
    s["out"] = torch.empty_like(s["q"])
    if own:
        import megatron_tensor_block_gb300 as tb
        s["plan"] = tb.tp_plan(dict(hidden=case["heads"] * d, n_heads=case["heads"], n_kv_heads=case["kv_heads"], head_dim=d,
                                    ffn=64 * n, n_experts=0, top_k=0, expert_ffn=0, org_vocab=0, eps=1e-5, rope_theta=5e5,
                                    dtype=tb.TP_BF16, has_qkv_bias=0, max_batch=case["batch"], max_tokens=tokens, max_kv=rows,
                                    expert_parallel=0), n)
        s["bytes"] = tb.tp_plan_get_info(s["plan"])["workspace_bytes"]
        s["workspace"] = torch.empty(s["bytes"], dtype=torch.uint8, device=dev)
        tb.tp_workspace_init(s["plan"], s["workspace"], s["bytes"])
    return s


def _prepare_logits(case, g, dev):
    history, prompt, bias, mask_row = _logit_lens(case)
    rows, vocab = case["rows"], case["vocab"]
    rand = lambda *shape: torch.rand(*shape, generator=g, device=dev)  # noqa: E731
    s = {"case": case, "logits": 3 * torch.randn(rows, vocab, generator=g, device=dev)}
    # a history repeats its own tokens, and common ones, more than rare ones
    s["tokens"] = (vocab * rand(sum(history)) ** 4).long().clamp_(max=vocab - 1).to(torch.int32)
    s["cu_tokens"], s["n_prompt"] = _cumulative(history, dev), torch.tensor(prompt, device=dev, dtype=torch.int32)
    s["repetition"], s["presence"], s["frequency"] = 1 + 0.5 * rand(rows), rand(rows) - 0.2, rand(rows) - 0.2
    if case["max_bias"]:
        s["bias_ids"] = torch.randint(0, vocab, (sum(bias),), generator=g, device=dev, dtype=torch.int32)
        s["bias_values"] = 10 * torch.randn(sum(bias), generator=g, device=dev)
        s["cu_bias"] = _cumulative(bias, dev)
    if case["masks"]:
        words = (vocab + 31) // 32
        draws = torch.randint(-(1 << 31), 1 << 31, (2, case["masks"], words), generator=g, device=dev)
        s["mask"] = (draws[0] & draws[1]).to(torch.int32)       # a quarter of the tokens allowed
        s["mask_row"] = torch.tensor(mask_row, device=dev, dtype=torch.int32)
    s["out"] = torch.empty_like(s["logits"])
    if own:
        import megatron_tensor_block_gb300 as tb
        s["plan"] = tb.tp_plan(dict(hidden=64, n_heads=1, n_kv_heads=1, head_dim=64, ffn=64, n_experts=0, top_k=0, expert_ffn=0,
                                    org_vocab=vocab, eps=1e-5, rope_theta=5e5, dtype=tb.TP_BF16, has_qkv_bias=0, max_batch=1,
                                    max_tokens=1, max_kv=1, expert_parallel=0), 1)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        import megatron_tensor_block_gb300 as tb
        if op == "packed":
            tb.tp_attn_packed(s["plan"], s["q"], (s["k"], s["v"]), s["cu"], s["pos"], s["case"]["batch"], s["tokens"], s["out"],
                              s["workspace"], s["bytes"])
        elif op == "prefix":
            tb.tp_attn_prefix(s["plan"], s["q"], (s["pk"], s["pv"]), s["case"]["prefix"], s["case"]["prefix"], (s["k"], s["v"]),
                              s["cu"], s["pos"], s["case"]["batch"], s["tokens"], s["out"], s["workspace"], s["bytes"])
        else:
            tb.tp_logits_process(s["plan"], s["logits"], s["case"]["rows"], s["out"], tokens=s["tokens"], cu_tokens=s["cu_tokens"],
                                 n_prompt=s["n_prompt"], repetition=s["repetition"], presence=s["presence"],
                                 frequency=s["frequency"], bias_ids=s.get("bias_ids"), bias_values=s.get("bias_values"),
                                 cu_bias=s.get("cu_bias"), mask=s.get("mask"), mask_row=s.get("mask_row"))
        return s["out"]
    return _plain_logits(s) if op == "logits" else _plain_attention(s)


def _plain_attention(s):
    """softmax(q k^T / sqrt(d)) v of every query head over its KV head's prefix and causal cache rows, the batch
    padded to its longest sequence."""
    case, q, dev = s["case"], s["q"], s["q"].device
    n, tokens, heads, d = q.shape
    b, m, rows, kv = case["batch"], s["longest"], s["rows"], case["kv_heads"] // case["tp"]
    cu, pos = s["cu"].long(), s["pos"].long()
    place = torch.arange(m, device=dev)
    at = (cu[:-1, None] + place).clamp_(max=tokens - 1)                                  # [b, m]: token of each padded row
    qs = q[:, at.view(-1)].float().view(n, b, m, kv, heads // kv, d).permute(0, 1, 3, 4, 2, 5) * d ** -0.5
    qs = qs.reshape(n, b, kv, heads // kv * m, d)
    k, v = torch.stack(s["k"]).float(), torch.stack(s["v"]).float()                      # [n, b, kv, rows, d]
    score = (qs @ k.transpose(-1, -2)).view(n, b, kv, heads // kv, m, rows)
    hidden = torch.arange(rows, device=dev) > (pos[:, None] + place)[..., None]          # [b, m, rows]
    score.masked_fill_(hidden[None, :, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if case["op"] == "prefix":
        pk, pv = torch.stack(s["pk"]).float(), torch.stack(s["pv"]).float()              # [n, kv, prefix, d]
        qp = qs.transpose(1, 2).reshape(n, kv, -1, d)
        far = (qp @ pk.transpose(-1, -2)).view(n, kv, b, heads // kv, m, -1).transpose(1, 2)
        top = torch.maximum(top, far.amax(-1, keepdim=True))
        far = far.sub_(top).exp_()
        near = score.sub_(top).exp_()
        total = near.sum(-1, keepdim=True) + far.sum(-1, keepdim=True)
        o = (far.transpose(1, 2).reshape(n, kv, -1, case["prefix"]) @ pv).view(n, kv, b, heads // kv, m, d).transpose(1, 2)
        o = o + (near.view(n, b, kv, -1, rows) @ v).view(n, b, kv, heads // kv, m, d)
    else:
        near = score.sub_(top).exp_()
        total = near.sum(-1, keepdim=True)
        o = (near.view(n, b, kv, -1, rows) @ v).view(n, b, kv, heads // kv, m, d)
    o = (o / total).permute(0, 1, 4, 2, 3, 5).reshape(n, b * m, heads, d)
    seq = torch.searchsorted(cu[1:], torch.arange(tokens, device=dev), right=True)
    return o[:, seq * m + torch.arange(tokens, device=dev) - cu[seq]].to(torch.bfloat16)


def _plain_logits(s):
    """Penalties of the tokens a row has seen, then its biases (the last of a token's counts), then its mask."""
    case, x, dev = s["case"], s["logits"], s["logits"].device
    rows, vocab = x.shape
    cu = s["cu_tokens"].long()
    at = torch.arange(s["tokens"].numel(), device=dev)
    row = torch.searchsorted(cu[1:], at, right=True)
    generated = (at - cu[row] >= s["n_prompt"].long()[row]).to(torch.int32)
    cell = row * vocab + s["tokens"].long()
    count = torch.zeros(rows * vocab, dtype=torch.int32, device=dev)
    seen = count.clone().index_add_(0, cell, torch.ones_like(generated)).view(rows, vocab) > 0
    count = count.index_add_(0, cell, generated).view(rows, vocab)
    r = s["repetition"][:, None]
    y = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    y = y - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if "bias_ids" in s:
        cu = s["cu_bias"].long()
        at = torch.arange(s["bias_ids"].numel(), device=dev)
        row = torch.searchsorted(cu[1:], at, right=True)
        last = torch.zeros(rows * vocab, dtype=torch.int64, device=dev)
        last.scatter_reduce_(0, row * vocab + s["bias_ids"].long(), at + 1, "amax")
        values = torch.cat([torch.zeros(1, device=dev), s["bias_values"]])
        y = y + values[last].view(rows, vocab)
    if "mask" in s:
        ids = torch.arange(vocab, device=dev)
        pick = s["mask_row"].long()
        allowed = (s["mask"][pick.clamp(min=0)][:, ids // 32] >> (ids % 32).to(torch.int32)) & 1
        y = y.masked_fill((allowed == 0) & (pick >= 0)[:, None], -math.inf)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_logits(s) if case["op"] == "logits" else _exact_attention(s)


def _exact_attention(s):
    case, q = s["case"], s["q"]
    new, cached = _lens(case)
    n, tokens, heads, d = q.shape
    kv, prefix = case["kv_heads"] // case["tp"], case.get("prefix", 0)
    group, out, first = heads // kv, torch.empty(q.shape, dtype=torch.float64, device=q.device), 0
    for b in range(case["batch"]):
        keys = torch.stack([t[b, :, :new[b] + cached[b]] for t in s["k"]])
        values = torch.stack([t[b, :, :new[b] + cached[b]] for t in s["v"]])
        if prefix:
            keys = torch.cat([torch.stack(s["pk"]), keys], 2)
            values = torch.cat([torch.stack(s["pv"]), values], 2)
        keys, values = keys.double(), values.double()
        step = max(1, int(2e8) // (n * heads * keys.shape[2]))
        for i in range(0, new[b], step):
            j = min(i + step, new[b])
            seen = prefix + cached[b] + j
            x = q[:, first + i:first + j].double().view(n, j - i, kv, group, d)
            w = torch.einsum("nikgd,nkld->nkgil", x, keys[:, :, :seen]) / math.sqrt(d)
            limit = prefix + cached[b] + torch.arange(i, j, device=q.device)
            w = torch.where(torch.arange(seen, device=q.device) <= limit[:, None], w, -math.inf)
            w = torch.exp(w - torch.logsumexp(w, -1, keepdim=True))
            out[:, first + i:first + j] = torch.einsum("nkgil,nkld->nikgd", w, values[:, :, :seen]).reshape(n, j - i, heads, d)
        first += new[b]
    return out


def _exact_logits(s):
    case = s["case"]
    history, prompt, bias, mask_row = _logit_lens(case)
    vocab, y = case["vocab"], s["logits"].double()
    first = start = 0
    for t in range(case["rows"]):
        ids = s["tokens"][first:first + history[t]].long()
        first += history[t]
        seen = torch.unique(ids)
        factor = s["repetition"][t].double()
        y[t, seen] = torch.where(y[t, seen] > 0, y[t, seen] / factor, y[t, seen] * factor)
        ids, times = torch.unique(ids[prompt[t]:], return_counts=True)
        y[t, ids] -= s["frequency"][t].double() * times + s["presence"][t].double()
        if "bias_ids" in s:
            chosen = dict(zip(s["bias_ids"][start:start + bias[t]].tolist(), s["bias_values"][start:start + bias[t]].tolist()))
            start += bias[t]
            if chosen:
                y[t, list(chosen)] += torch.tensor(list(chosen.values()), dtype=torch.float64, device=y.device)
        if mask_row[t] >= 0:
            bits = (s["mask"][mask_row[t]].unsqueeze(1) >> torch.arange(32, device=y.device, dtype=torch.int32)) & 1
            y[t, bits.reshape(-1)[:vocab] == 0] = -math.inf
    return y
