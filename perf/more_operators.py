"""Cases, plain forms and 64-bit values of the operators around an 8-bit paged
KV cache of the tensor-parallel block library: the rotary embedding of a packed
batch in its layouts and scalings (``tp_rope_packed``), appending the batch's
keys and values to the pages with that rotation on the way
(``tp_kv_append_paged``), and the attention that reads the pages
(``tp_attn_paged``).

A cache page holds ``page`` tokens of every KV head of a shard as e4m3 values,
and a scale, a power of two, for each page and head. Head layouts and shard
counts are those of the workloads in ``synth.py``; the others are generic.
"""
import math
import random

import torch

own = False

# (query heads, KV heads, head size, shards): the Llama-3-8B-shaped and Qwen2.5-0.5B-shaped layers of synth.py
LLAMA_TP8 = dict(heads=32, kv_heads=8, head_dim=128, tp=8)
LLAMA_TP4 = dict(heads=32, kv_heads=8, head_dim=128, tp=4)
QWEN_TP2 = dict(heads=14, kv_heads=2, head_dim=64, tp=2)

# rotations: layout 0 pairs features i and i + rot / 2, layout 1 features 2 i and 2 i + 1; scaling 0 none, 1 linear,
# 2 by wavelength, 3 by a ramp over the pairs with a factor on the result
PLAIN = dict(rot=0, layout=0, scaling=0, theta=1e6, factor=1.0, low=0.0, high=0.0, original=0)
WAVES = dict(rot=0, layout=0, scaling=2, theta=5e5, factor=8.0, low=1.0, high=4.0, original=8192)
RAMP = dict(rot=0, layout=0, scaling=3, theta=1e6, factor=4.0, low=1.0, high=32.0, original=32768)
PARTIAL = dict(rot=32, layout=1, scaling=1, theta=1e4, factor=2.0, low=0.0, high=0.0, original=0)

MIN_EXPONENT = -60          # of a page's scale
TOP = 448.0                 # the largest e4m3 value


def _case(name, op, layout, rope, page, batch, min_new, max_new, min_cached, max_cached, lens_seed):
    return {"name": name, "op": op, **layout, **rope, "page": page, "batch": batch, "min_new": min_new, "max_new": max_new,
            "min_cached": min_cached, "max_cached": max_cached, "lens_seed": lens_seed}


def listed():
    return [
        # rotating the new tokens of a decode step of 64 chats: latency
        _case("rope_decode_64", "rope", LLAMA_TP4, WAVES, 0, 64, 1, 1, 0, 100000, 1),
        # a prefill batch of a model with interleaved pairs that rotates half of each head
        _case("rope_partial_interleaved", "rope", QWEN_TP2, PARTIAL, 0, 9, 1, 1024, 0, 4096, 2),
        # a long document, its context stretched
        _case("rope_long_prompt", "rope", LLAMA_TP8, RAMP, 0, 1, 16384, 16384, 0, 0, 3),
        # one new token of one sequence: the smallest call, all latency
        _case("append_one_token", "append", QWEN_TP2, PLAIN, 16, 1, 1, 1, 512, 512, 4),
        # the decode step of a busy server: one token each, most of them in the middle of a page
        _case("append_decode_256", "append", LLAMA_TP4, WAVES, 64, 256, 1, 1, 0, 255, 5),
        # prompts of unlike lengths, some continuing a page that earlier turns have filled in part
        _case("append_prompts", "append", LLAMA_TP8, WAVES, 32, 24, 1, 2048, 0, 100, 6),
        # the attention of one token of one sequence over a cache of 512: latency
        _case("attend_one_token", "attend", QWEN_TP2, PLAIN, 16, 1, 1, 1, 512, 512, 7),
        # a decode step of 64 chats of unlike lengths
        _case("attend_decode_64", "attend", LLAMA_TP4, PLAIN, 64, 64, 1, 1, 256, 4095, 8),
        # a decode step of many long contexts: the bytes of the cache
        _case("attend_decode_128_long", "attend", LLAMA_TP4, PLAIN, 128, 128, 1, 1, 1, 16383, 9),
        # drafted tokens to be verified: a few new tokens for each sequence
        _case("attend_drafted", "attend", LLAMA_TP8, PLAIN, 16, 32, 1, 8, 100, 4000, 10),
        # a prefill batch of unlike prompts, some behind cached turns
        _case("attend_prompts", "attend", LLAMA_TP8, PLAIN, 32, 12, 1, 2048, 0, 500, 11),
        # one chunk of a long prompt that is prefilled piece by piece
        _case("attend_chunk_of_long", "attend", LLAMA_TP4, PLAIN, 128, 1, 512, 512, 30001, 30001, 12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "append", "append", "attend", "attend", "attend"])
        group, kv = rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 128])
        layout = rng.choice([QWEN_TP2, LLAMA_TP4, LLAMA_TP8,
                             dict(heads=group * kv, kv_heads=kv, head_dim=d, tp=rng.choice([t for t in (1, 2, 4, 8) if kv % t == 0]))])
        rope = dict(rng.choice([PLAIN, WAVES, RAMP, PARTIAL]))
        if op != "attend":
            rope["layout"], rope["rot"] = rng.choice([0, 1]), rng.choice([0, 0, 16, 32, 64])
        batch = _log_int(rng, 1, 256)
        most = rng.choice([1, 1, _log_int(rng, 1, 8), _log_int(rng, 1, 4096)])
        cached = rng.choice([0, _log_int(rng, 1, 16384 if op == "attend" else 300)])
        c = {"op": op, **layout, **rope, "page": 0 if op == "rope" else rng.choice([16, 32, 64, 128]), "batch": batch,
             "min_new": 1 if batch > 1 else max(1, most // 2), "max_new": most, "min_cached": 0, "max_cached": cached,
             "lens_seed": rng.randint(100, 1 << 30)}
        new, old = _lens(c)
        # the plain form pads every sequence to the longest: keep its scores, and its copies of the keys, of a size it can hold
        scores = batch * c["heads"] * max(new) * (most + cached)
        keys = batch * c["kv_heads"] * (max(new) + max(old)) * c["head_dim"]
        w = work(c)
        if op == "attend" and w["flops"] <= 2.5e11 and w["bytes"] <= 1.5e9 and scores <= 2e9 and keys <= 1.2e9:
            return c
        if op != "attend" and sum(new) * c["heads"] * c["head_dim"] <= 16384 * 4096 and keys <= 1e8:
            return c


def _lens(case):
    """Lengths of a batch, from the case alone: (new tokens, cached tokens) of every sequence."""
    rng = random.Random(case["lens_seed"])
    new = [_log_int(rng, case["min_new"], case["max_new"]) for _ in range(case["batch"])]
    cached = [rng.randint(case["min_cached"], case["max_cached"]) for _ in range(case["batch"])]
    return new, cached


def work(case):
    new, cached = _lens(case)
    d, heads, kv_heads, tokens = case["head_dim"], case["heads"], case["kv_heads"], sum(new)
    if case["op"] == "rope":
        turned = tokens * (heads + kv_heads) * (case["rot"] or d)
        return {"bytes": 4 * tokens * (heads + kv_heads) * d, "flops": 3 * turned}
    if case["op"] == "append":
        pages = sum((c + n - 1) // case["page"] - c // case["page"] + 1 for n, c in zip(new, cached))
        return {"bytes": tokens * d * (4 * heads + 2 * kv_heads * 3) + 8 * pages * kv_heads,
                "flops": 3 * tokens * (heads + kv_heads) * (case["rot"] or d) + 2 * tokens * kv_heads * d}
    seen = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, cached))
    keys = sum(n + c for n, c in zip(new, cached))
    pages = sum(-(-(n + c) // case["page"]) for n, c in zip(new, cached))
    return {"bytes": 4 * tokens * heads * d + 2 * keys * kv_heads * d + pages * (8 * kv_heads + 4), "flops": 4 * d * heads * seen}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    new, cached = _lens(case)
    n, heads, kv, d = case["tp"], case["heads"] // case["tp"], case["kv_heads"] // case["tp"], case["head_dim"]
    tokens, op = sum(new), case["op"]

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    s = {"case": case, "tokens": tokens, "longest": max(new), "rows": max(a + b for a, b in zip(new, cached))}
    s["cu"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    s["pos"] = torch.tensor(cached, device=dev, dtype=torch.int32)
    # queries of some heads are sharper than others', and some features of a key larger than others, as in a trained layer
    sharp = 0.5 + 1.5 * torch.rand(n, 1, heads, 1, generator=g, device=dev)
    gain = torch.exp(0.5 * normal(n, 1, kv, d, dtype=torch.float32))
    s["q"] = (normal(n, tokens, heads, d) * sharp).to(torch.bfloat16)
    s["q_out"] = torch.empty_like(s["q"])
    if op != "attend":
        s["k"] = (normal(n, tokens, kv, d) * gain).to(torch.bfloat16)
        s["k_out"] = torch.empty_like(s["k"])
    if op != "rope":
        page = case["page"]
        need = [-(-(a + b) // page) for a, b in zip(new, cached)]
        pages = sum(need) + 3                                                       # a few of the pool's are free
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        s["table"] = torch.full((case["batch"], max(need)), -1, device=dev, dtype=torch.int32)
        first = 0
        for b, m in enumerate(need):
            s["table"][b, :m] = order[first:first + m]
            first += m
        for name, by in (("k", gain), ("v", torch.exp(0.5 * normal(n, 1, kv, 1, dtype=torch.float32)))):
            s["pool_" + name] = torch.empty(n, pages, kv, page, d, device=dev, dtype=torch.float8_e4m3fn)
            s["scale_" + name] = torch.empty(n, pages, kv, device=dev)
            some = max(1, (1 << 26) // (kv * page * d))
            for r in range(n):
                for i in range(0, pages, some):                                     # what earlier calls have stored
                    x = normal(min(some, pages - i), kv, page, d, dtype=torch.float32) * by[r, :, :, None]
                    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((-2, -1)) / TOP)))
                    s["scale_" + name][r, i:i + some] = scale
                    s["pool_" + name][r, i:i + some] = (x / scale[..., None, None]).to(torch.float8_e4m3fn)
    if op == "append":
        s["v"] = normal(n, tokens, kv, d)
    if op == "attend":
        s["out"] = torch.empty_like(s["q"])
    if own:
        import megatron_tensor_block_gb300 as tb
        s["plan"] = tb.tp_plan(dict(hidden=case["heads"] * d, n_heads=case["heads"], n_kv_heads=case["kv_heads"], head_dim=d,
                                    ffn=64 * n, n_experts=0, top_k=0, expert_ffn=0, org_vocab=0, eps=1e-5, rope_theta=case["theta"],
                                    dtype=tb.TP_BF16, has_qkv_bias=0, max_batch=case["batch"], max_tokens=tokens, max_kv=s["rows"],
                                    expert_parallel=0), n)
        s["rope"] = tb.tp_rope(rot_dim=case["rot"], layout=case["layout"], scaling=case["scaling"], theta=case["theta"],
                               factor=case["factor"], low=case["low"], high=case["high"], original=case["original"])
        if op != "rope":
            s["kv"] = tb.PagedKV(s["plan"], list(s["pool_k"]), list(s["pool_v"]), list(s["scale_k"]), list(s["scale_v"]), s["table"])
        if op == "attend":
            s["bytes"] = tb.tp_paged_workspace_bytes(s["plan"])
            s["workspace"] = torch.empty(s["bytes"], dtype=torch.uint8, device=dev)
            tb.tp_paged_workspace_init(s["plan"], s["workspace"], s["bytes"])
    return s


def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        import megatron_tensor_block_gb300 as tb
        if op == "rope":
            tb.tp_rope_packed(s["plan"], s["rope"], s["cu"], s["pos"], case["batch"], s["tokens"], q=s["q"], q_out=s["q_out"],
                              k=s["k"], k_out=s["k_out"])
        elif op == "append":
            tb.tp_kv_append_paged(s["plan"], s["rope"], s["k"], s["v"], s["kv"], s["cu"], s["pos"], case["batch"], s["tokens"],
                                  q=s["q"], q_out=s["q_out"])
        else:
            tb.tp_attn_paged(s["plan"], s["q"], s["kv"], s["cu"], s["pos"], case["batch"], s["tokens"], s["out"], s["workspace"],
                             s["bytes"], max_new=s["longest"])
            return s["out"]
    elif op == "attend":
        return _plain_attention(s)
    else:
        turn = _plain_turn(s)
        s["q_out"] = turn(s["q"].double()).to(torch.bfloat16)
        if op == "append":
            _plain_append(s, turn(s["k"].double()))
        else:
            s["k_out"] = turn(s["k"].double()).to(torch.bfloat16)
    if op == "rope":
        return {"q": s["q_out"], "k": s["k_out"]}
    return {"q": s["q_out"], "k": s["pool_k"], "v": s["pool_v"], "k_scale": s["scale_k"], "v_scale": s["scale_v"]}


def _tokens(s):
    """(sequence, position) of every token row."""
    cu, at = s["cu"].long(), torch.arange(s["tokens"], device=s["cu"].device)
    seq = torch.searchsorted(cu[1:], at, right=True)
    return seq, s["pos"].long()[seq] + at - cu[seq]


def _plain_turn(s):
    """The rotation of rows [shards, tokens, heads, d] in 64 bits: angles of far positions lose all their digits in 32."""
    case, dev = s["case"], s["q"].device
    rot = case["rot"] or case["head_dim"]
    i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
    f, by = case["theta"] ** (-2 * i / rot), 1.0
    if case["scaling"] == 1:
        f = f / case["factor"]
    elif case["scaling"] == 2:
        turns = case["original"] * f / (2 * math.pi)
        f = f / case["factor"] + (f - f / case["factor"]) * ((turns - case["low"]) / (case["high"] - case["low"])).clamp(0, 1)
    elif case["scaling"] == 3:
        edge = [rot * math.log(case["original"] / (2 * math.pi * b)) / (2 * math.log(case["theta"])) for b in (case["high"], case["low"])]
        first, last = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
        slow = ((i - first) / max(last - first, 0.001)).clamp(0, 1)
        f = f * (1 - slow) + f / case["factor"] * slow
        by = 0.1 * math.log(case["factor"]) + 1
    angle = _tokens(s)[1].double()[:, None, None] * f
    cos, sin = by * angle.cos(), by * angle.sin()

    def turn(x):
        y = x.clone()
        a = slice(0, rot // 2) if case["layout"] == 0 else slice(0, rot, 2)
        b = slice(rot // 2, rot) if case["layout"] == 0 else slice(1, rot, 2)
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., a] * sin + x[..., b] * cos
        return y

    return turn


def _key_growth(case):
    """How much a turned pair's features may exceed the larger of the two: the scale of a page goes by it."""
    return math.sqrt(2.0) * (max(1.0, 0.1 * math.log(case["factor"]) + 1) if case["scaling"] == 3 else 1.0)


def _plain_append(s, turned):
    """Every page that a new token falls into: its scale raised to what the new values need (taken anew where its first
    slot is written), the stored values brought to it, the new ones rounded to e4m3 by it."""
    case, page = s["case"], s["case"]["page"]
    seq, pos = _tokens(s)
    at, slot = s["table"][seq, pos // page].long(), pos % page
    for name, new, given, growth in (("k", turned, s["k"], _key_growth(case)), ("v", s["v"].double(), s["v"], 1.0)):
        pool, scale = s["pool_" + name], s["scale_" + name]
        most = given.double().abs().amax(-1) * growth / TOP                                     # [n, tokens, kv]
        need = torch.zeros(scale.shape, dtype=torch.float64, device=scale.device).index_reduce_(1, at, most, "amax")
        power = torch.ceil(torch.log2(need)).clamp_(min=MIN_EXPONENT)
        power = power + (torch.exp2(power) < need).double()
        power = power - ((torch.exp2(power - 1) >= need) & (power > MIN_EXPONENT)).double()
        touched = torch.zeros(scale.shape[1], dtype=torch.bool, device=scale.device).index_fill_(0, at, True)
        fresh = torch.zeros_like(touched).index_fill_(0, at[slot == 0], True)
        raised = torch.where(fresh[:, None], torch.exp2(power), torch.maximum(scale.double(), torch.exp2(power)))
        after = torch.where(touched[:, None], raised, scale.double())
        # what a page that is begun anew still holds behind the new tokens is another sequence's: it stays as it is
        again = pool.float().double() * torch.where(fresh[:, None], 1.0, scale.double() / after)[..., None, None]
        again[:, at, :, slot] = (new / after[:, at][..., None]).transpose(0, 1)
        pool.copy_(_e4m3(again))
        scale.copy_(after.float())


def _e4m3(x):
    """Values within +-448 to the nearest with four significant bits, 2^-9 apart at least; ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs())).clamp_(min=-6) - 3)
    return (torch.round(x / step) * step).float().to(torch.float8_e4m3fn)


def _plain_attention(s):
    """softmax(q k^T / sqrt(d)) v of every query head over its sequence's pages, brought back to 32 bits, the batch
    padded to its longest sequence."""
    case, q, dev = s["case"], s["q"], s["q"].device
    n, tokens, heads, d = q.shape
    b, m, kv = case["batch"], s["longest"], case["kv_heads"] // case["tp"]
    cu, pos, table = s["cu"].long(), s["pos"].long(), s["table"].long()
    rows = table.shape[1] * case["page"]
    place = torch.arange(m, device=dev)
    at = (cu[:-1, None] + place).clamp_(max=tokens - 1)                                  # [b, m]: token of each padded row
    qs = q[:, at.view(-1)].float().view(n, b, m, kv, heads // kv, d).permute(0, 1, 3, 4, 2, 5) * d ** -0.5
    qs = qs.reshape(n, b, kv, heads // kv * m, d)

    def cache(name):                                                                     # [n, b, kv, rows, d]
        x = s["pool_" + name].view(torch.uint8)[:, table.clamp(min=0)].view(torch.float8_e4m3fn).float()
        x *= s["scale_" + name][:, table.clamp(min=0)][..., None, None]
        return x.transpose(2, 3).reshape(n, b, kv, rows, d)

    score = (qs @ cache("k").transpose(-1, -2)).view(n, b, kv, heads // kv, m, rows)
    hidden = torch.arange(rows, device=dev) > (pos[:, None] + place)[..., None]          # [b, m, rows]
    score.masked_fill_(hidden[None, :, None, None], -math.inf)
    weight = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = weight.sum(-1, keepdim=True)
    o = (weight.view(n, b, kv, -1, rows) @ cache("v")).view(n, b, kv, heads // kv, m, d) / total
    o = o.permute(0, 1, 4, 2, 3, 5).reshape(n, b * m, heads, d)
    seq = _tokens(s)[0]
    return o[:, seq * m + torch.arange(tokens, device=dev) - cu[seq]].to(torch.bfloat16)


def exact(case, seed):
    """As ``run``, without any rounding: stored values are those that the rounding to e4m3 is nearest to."""
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attention(s)
    new, cached = _lens(case)
    rot = case["rot"] or case["head_dim"]
    speeds, by = [], 1.0
    for i in range(rot // 2):
        f = math.exp(-2 * i / rot * math.log(case["theta"]))
        if case["scaling"] == 1:
            f /= case["factor"]
        elif case["scaling"] == 2:
            wave = 2 * math.pi / f
            if wave > case["original"] / case["low"]:
                f /= case["factor"]
            elif wave > case["original"] / case["high"]:
                mix = (case["original"] / wave - case["low"]) / (case["high"] - case["low"])
                f = (1 - mix) * f / case["factor"] + mix * f
        elif case["scaling"] == 3:
            def pair(turns):                    # the pair that turns so often over the original length
                return rot / 2 * math.log(case["original"] / (turns * 2 * math.pi)) / math.log(case["theta"])
            lo, hi = max(math.floor(pair(case["high"])), 0), min(math.ceil(pair(case["low"])), rot - 1)
            share = min(1.0, max(0.0, (i - lo) / ((hi - lo) or 0.001)))
            f = share * f / case["factor"] + (1 - share) * f
            by = 1 + math.log(case["factor"]) / 10
        speeds.append(f)
    where = torch.cat([torch.arange(c, c + n, dtype=torch.float64) for n, c in zip(new, cached)]).to(s["q"].device)
    spin = by * torch.exp(1j * where[:, None] * torch.tensor(speeds, dtype=torch.float64, device=where.device))

    def turn(x):
        x = x.double()
        pairs = x[..., :rot].unflatten(-1, (2, rot // 2)).movedim(-2, -1) if case["layout"] == 0 else x[..., :rot].unflatten(-1, (rot // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * spin[:, None])
        z = z.movedim(-1, -2) if case["layout"] == 0 else z
        return torch.cat([z.flatten(-2), x[..., rot:]], -1)

    if case["op"] == "rope":
        return {"q": turn(s["q"]), "k": turn(s["k"])}
    out = {"q": turn(s["q"])}
    table = s["table"].tolist()
    for name, values, growth in (("k", turn(s["k"]), _key_growth(case)), ("v", s["v"].double(), 1.0)):
        pool, scale = s["pool_" + name].float().double(), s["scale_" + name].double()
        first = 0
        for b in range(case["batch"]):
            t = 0
            while t < new[b]:
                slot = (cached[b] + t) % case["page"]
                count = min(case["page"] - slot, new[b] - t)
                at, rows = table[b][(cached[b] + t) // case["page"]], slice(first + t, first + t + count)
                size = s[name][:, rows].double().abs().amax((1, 3)) * growth / TOP
                half, power = torch.frexp(size)
                power = torch.where(half == 0.5, power - 1, power).clamp(min=MIN_EXPONENT)
                power = torch.where(size == 0, MIN_EXPONENT, power)
                wanted = torch.pow(2.0, power.double())
                if slot:
                    wanted = torch.maximum(wanted, scale[:, at])
                    pool[:, at] *= (scale[:, at] / wanted)[..., None, None]
                scale[:, at] = wanted
                pool[:, at, :, slot:slot + count] = values[:, rows].transpose(1, 2) / wanted[..., None, None]
                t += count
            first += new[b]
        out[name], out[name + "_scale"] = pool, scale
    return out


def _exact_attention(s):
    case, q = s["case"], s["q"]
    new, cached = _lens(case)
    n, tokens, heads, d = q.shape
    kv, page = case["kv_heads"] // case["tp"], case["page"]
    group, out, first = heads // kv, torch.empty(q.shape, dtype=torch.float64, device=q.device), 0
    for b in range(case["batch"]):
        end = new[b] + cached[b]
        ids = s["table"][b, :-(-end // page)].long()

        def read(name):
            x = s["pool_" + name].view(torch.uint8)[:, ids].view(torch.float8_e4m3fn).float().double()
            x *= s["scale_" + name][:, ids].double()[..., None, None]
            return x.transpose(1, 2).flatten(2, 3)[:, :, :end]

        keys, values = read("k"), read("v")
        step = max(1, int(2e8) // (n * heads * end))
        for i in range(0, new[b], step):
            j = min(i + step, new[b])
            seen = cached[b] + j
            x = q[:, first + i:first + j].double().view(n, j - i, kv, group, d)
            w = torch.einsum("nikgd,nkld->nkgil", x, keys[:, :, :seen]) / math.sqrt(d)
            limit = cached[b] + torch.arange(i, j, device=q.device)
            w = torch.where(torch.arange(seen, device=q.device) <= limit[:, None], w, -math.inf)
            w = torch.exp(w - torch.logsumexp(w, -1, keepdim=True))
            out[:, first + i:first + j] = torch.einsum("nkgil,nkld->nikgd", w, values[:, :, :seen]).reshape(n, j - i, heads, d)
        first += new[b]
    return out
