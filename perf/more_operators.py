"""A server's step over the paged Q8_0 cache, around and beside its attention: slots and block tables from request
lengths, norms of queries and keys with their rotary positions, attention in a sliding window with sinks, and attention
of a batch behind a shared prefix; with plain forms of the same operators.

Q8_0 rows: a head row of D channels is D / 32 blocks of 34 bytes, an fp16 scale d and 32 int8 codes c; its values are
d * c.  Pages: uint8 [n_pages][kv_heads][page_tokens][D / 32 * 34]; a row's slot is page * page_tokens + offset.
"""

import math

import torch

own = False

_F16, _BF16, _F32 = "float16", "bfloat16", "float32"


def listed():
    return [
        # the tables of one step of 64 sequences, a token each: latency
        {"name": "extend_step", "op": "extend", "batch": 64, "max_new": 1, "min_new": 1, "max_kv": 16384, "page": 64,
         "padding": 0},
        # a step of 1,000 sequences, bursts of up to 16 candidates, padded to a captured size
        {"name": "extend_bursts", "op": "extend", "batch": 1000, "max_new": 16, "min_new": 0, "max_kv": 32768,
         "page": 16, "padding": 500},
        # prompts of 31 to 8,192 tokens enter
        {"name": "extend_prompts", "op": "extend", "batch": 48, "max_new": 8192, "min_new": 31, "max_kv": 0,
         "page": 16, "padding": 0},
        # the queries and keys of one step of 64 sequences, slices of the fused projection's output
        {"name": "norm_step", "op": "norm_rope", "tokens": 64, "heads": 32, "kv_heads": 8, "d": 128, "rot": 128,
         "axes": 1, "interleaved": False, "dtype": _BF16, "norm": True, "max_pos": 65536, "packed": True},
        # those of a prompt of 16,384 tokens
        {"name": "norm_prompt", "op": "norm_rope", "tokens": 16384, "heads": 32, "kv_heads": 8, "d": 128, "rot": 128,
         "axes": 1, "interleaved": False, "dtype": _BF16, "norm": True, "max_pos": 1048576, "packed": True},
        # 9,001 patches of a video with positions in time, height and width, pairs of neighbouring channels
        {"name": "norm_video", "op": "norm_rope", "tokens": 9001, "heads": 24, "kv_heads": 24, "d": 64, "rot": 64,
         "axes": 3, "interleaved": True, "dtype": _F16, "norm": True, "max_pos": 4096, "packed": True},
        # one new token after 131,071, of which it sees the last 1,024 and the first 4: latency
        {"name": "window_one", "op": "window", "batch": 1, "max_q": 1, "min_q": 1, "max_kv": 131071, "min_kv": 131071,
         "heads": 32, "kv_heads": 8, "d": 64, "page": 64, "dtype": _F16, "window": 1024, "sinks": 4},
        # one new token for each of 64 sequences of very different lengths, windows of 4,096
        {"name": "window_batch", "op": "window", "batch": 64, "max_q": 1, "min_q": 1, "max_kv": 65536, "min_kv": 300,
         "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "dtype": _BF16, "window": 4096, "sinks": 4},
        # whole prompts in windows of 4,000
        {"name": "window_prompt", "op": "window", "batch": 3, "max_q": 8192, "min_q": 3001, "max_kv": 0, "min_kv": 0,
         "heads": 32, "kv_heads": 8, "d": 128, "page": 128, "dtype": _F16, "window": 4000, "sinks": 16},
        # one new token for each of four sequences behind a short shared prompt: latency
        {"name": "prefix_few", "op": "prefix", "batch": 4, "max_q": 1, "min_q": 1, "prefix": 2048, "max_own": 200,
         "min_own": 9, "heads": 32, "kv_heads": 8, "d": 64, "page": 16, "dtype": _F16},
        # one new token for each of 64 sequences behind a shared context of 32,768 tokens
        {"name": "prefix_batch", "op": "prefix", "batch": 64, "max_q": 1, "min_q": 1, "prefix": 32768, "max_own": 2048,
         "min_own": 100, "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "dtype": _BF16},
        # bursts of 2 to 8 candidates for each of 16 sequences behind 100,001 tokens, a context that ends inside a page
        {"name": "prefix_burst", "op": "prefix", "batch": 16, "max_q": 8, "min_q": 2, "prefix": 100001,
         "max_own": 1000, "min_own": 30, "heads": 32, "kv_heads": 8, "d": 64, "page": 128, "dtype": _F16},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["extend", "norm_rope", "norm_rope", "window", "window", "window", "prefix", "prefix"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "extend":
        batch = log_int(1, 2000)
        new = 1 if rng.random() < 0.3 else log_int(2, max(2, min(8192, 200000 // batch)))
        return {"op": op, "batch": batch, "max_new": new, "min_new": rng.choice([0, 1, new // 3]),
                "max_kv": rng.choice([0, log_int(10, 65536)]), "page": page, "padding": rng.choice([0, log_int(1, 500)])}
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 8])
    heads = min(32, kv_heads * rng.choice([1, 3, 4, 8]))
    if op == "norm_rope":
        axes = rng.choice([1, 1, 2, 3])
        return {"op": op, "tokens": log_int(1, 16384), "heads": heads, "kv_heads": kv_heads, "d": d,
                "rot": rng.choice([d, d, d // 2, d // 4]), "axes": axes, "interleaved": rng.random() < 0.4,
                "dtype": rng.choice([_F16, _BF16, _BF16, _F32]), "norm": rng.random() < 0.8,
                "max_pos": log_int(1000, 1 << 20) if axes == 1 else log_int(50, 5000), "packed": rng.random() < 0.5}
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "d": d, "page": page, "dtype": rng.choice([_F16, _BF16])}
    if op == "window":
        case.update(window=log_int(16, 6000), sinks=rng.choice([0, 1, 4, 16, log_int(17, 500)]))
        kind = rng.choice(["decode", "burst", "chunk", "whole"])
        if kind == "decode":
            batch = log_int(1, 64)
            hi = log_int(20, 65536)
            return {**case, "batch": batch, "max_q": 1, "min_q": 1, "max_kv": hi, "min_kv": max(1, hi // 9)}
        if kind == "burst":
            batch, q = log_int(1, 8), rng.randint(2, 64)
            hi = log_int(100, 65536)
            return {**case, "batch": batch, "max_q": q, "min_q": max(1, q // 2), "max_kv": hi, "min_kv": max(q, hi // 5)}
        if kind == "chunk":
            batch, q = rng.randint(1, 3), log_int(65, 2048)
            hi = q + log_int(50, 16384)
            return {**case, "batch": batch, "max_q": q, "min_q": max(1, q // 6), "max_kv": hi, "min_kv": q}
        batch, q = rng.randint(1, 3), log_int(30, 4500)
        return {**case, "batch": batch, "max_q": q, "min_q": max(1, q // 4), "max_kv": 0, "min_kv": 0}
    batch = log_int(2, 64)
    q = 1 if rng.random() < 0.6 else rng.randint(2, 16)
    own_keys = q + log_int(5, 2048)
    prefix = log_int(300, 100000 if batch <= 16 else 32768)
    return {**case, "batch": batch, "max_q": q, "min_q": max(1, q // 3), "prefix": prefix,
            "max_own": own_keys,
            "min_own": max(q, own_keys // 9)}


# ---------------------------------------------------------------- inputs --


def _spread(hi, lo, n, step=5):
    """n whole numbers from hi to lo, the first the largest, out of order."""
    return [hi - (hi - lo) * ((step * i) % n) // max(1, n - 1) for i in range(n)]


def _lengths(case):
    """(new tokens, keys with them) of each sequence."""
    n = case["batch"]
    q = _spread(case["max_q"], case["min_q"], n)
    if case["op"] == "prefix":
        return q, [case["prefix"] + max(m, a) for m, a in zip(_spread(case["max_own"], case["min_own"], n, 1), q)]
    return q, [max(m, a) for m, a in zip(_spread(case["max_kv"], case["min_kv"], n, 1), q)]


def _visible(case, nq, n):
    """(query, key) pairs of a sequence in its window, and the keys that any of its queries sees."""
    w, s = case["window"], case["sinks"]
    p = torch.arange(n - nq, n)
    low = (p - w + 1).clamp(min=0)
    pairs = int((p + 1 - low + low.clamp(max=s)).sum())
    first = int(low[0])
    return pairs, n - first + min(first, s)


def _random_pages(n_pages, kv_heads, page, d, gen):
    """Pages of quantised standard normal values."""
    out = torch.empty((n_pages, kv_heads, page, d // 32 * 34), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (kv_heads * page * d))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        x = torch.randn((n, kv_heads, page, d // 32, 32), generator=gen, device="cuda")
        scale = (x.abs().amax(-1, keepdim=True) / 127).half()
        codes = (x / scale.float()).round().clamp(-127, 127).to(torch.int8)
        out[i:i + n] = torch.cat([scale.view(torch.uint8), codes.view(torch.uint8)], -1).flatten(-2)
    return out


def _sections(pairs, axes):
    """Pairs of each axis: the first axis about half as many as the others."""
    first = pairs if axes == 1 else max(1, pairs // (2 * axes - 1))
    rest = [] if axes == 1 else [(pairs - first) // (axes - 1)] * (axes - 1)
    if rest:
        rest[-1] += pairs - first - sum(rest)
    return [first] + rest


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    page = case.get("page")
    if case["op"] == "extend":
        n = case["batch"]
        new = torch.tensor(_spread(case["max_new"], case["min_new"], n), device="cuda")
        new = new[torch.randperm(n, generator=gen, device="cuda")]
        kv = torch.randint(0, case["max_kv"] + 1, (n,), generator=gen, device="cuda")
        s["new_lens"], s["kv_lens"] = new.int(), kv.int()
        s["total"] = int(new.sum()) + case["padding"]
        had, have = -(-kv // page), -(-(kv + new) // page)
        n_pages = int(have.sum()) + 7
        order = torch.randperm(n_pages, generator=gen, device="cuda").int()
        width = -(-(case["max_kv"] + case["max_new"]) // page)
        at = torch.arange(width, device="cuda")
        first = had.cumsum(0) - had
        s["block_table"] = torch.where(at < had[:, None], order[(first[:, None] + at).clamp(max=n_pages - 1)], -1)
        s["free_pages"] = order[int(had.sum()):].contiguous()
        s["n_free"] = torch.tensor([len(s["free_pages"])], dtype=torch.int32, device="cuda")
        return s
    dtype = getattr(torch, case["dtype"])
    d, hq, hk = case["d"], case["heads"], case["kv_heads"]
    if case["op"] == "norm_rope":
        n, rot, axes = case["tokens"], case["rot"], case["axes"]
        i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = 10000.0 ** (-i / rot)
        if axes == 1:
            if n <= 256:   # a step: each token its own sequence's position
                s["positions"] = torch.randint(0, case["max_pos"], (1, n), generator=gen, device="cuda")
            else:
                start = torch.randint(0, max(1, case["max_pos"] - n), (1,), generator=gen, device="cuda")
                s["positions"] = (start + torch.arange(n, device="cuda"))[None]
        else:   # a grid: the last axis fastest
            side = max(1, round(n ** (1 / axes)))
            at = torch.arange(n, device="cuda")
            start = torch.randint(0, case["max_pos"], (axes, 1), generator=gen, device="cuda")
            grid = [at // side ** (axes - 1 - a) % (side if a else n) for a in range(axes)]
            s["positions"] = start + torch.stack(grid)
        s["axes"] = None
        if axes > 1:
            s["axes"] = torch.repeat_interleave(torch.arange(axes, device="cuda"),
                                                torch.tensor(_sections(rot // 2, axes), device="cuda")).int()
        make = lambda h: (torch.randn((n, h, d), generator=gen, device="cuda") * 1.7).to(dtype)
        if case["packed"]:   # queries, keys and values side by side
            s["q"], s["k"], _ = make(hq + 2 * hk).split([hq, hk, hk], dim=1)
        else:
            s["q"], s["k"] = make(hq), make(hk)
        weight = lambda: (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dtype)
        s["q_weight"], s["k_weight"] = (weight(), weight()) if case["norm"] else (None, None)
        return s
    q_len, kv_len = _lengths(case)
    shared = case["prefix"] // page if case["op"] == "prefix" else 0   # whole pages of the prefix
    used = [-(-n // page) - shared for n in kv_len]
    width = shared + max(used)
    n_pages = shared + sum(used) + 1
    s["k_pages"] = _random_pages(n_pages, hk, page, d, gen)
    s["v_pages"] = _random_pages(n_pages, hk, page, d, gen)
    order = torch.randperm(n_pages, generator=gen, device="cuda").int()
    s["block_table"] = torch.zeros((case["batch"], width), dtype=torch.int32, device="cuda")
    s["block_table"][:, :shared] = order[:shared]
    first = shared
    for b, n in enumerate(used):
        s["block_table"][b, shared:shared + n] = order[first:first + n]
        first += n
    if shared:
        # what is beyond the prefix's last whole page is each sequence's own, with the same contents
        rest = case["prefix"] % page
        own_first = s["block_table"][:, shared].long()
        for pool in (s["k_pages"], s["v_pages"]):
            pool[own_first, :, :rest] = pool[own_first[:1], :, :rest]
        s["prefix_table"] = s["block_table"][0, :-(-case["prefix"] // page)].clone()
        s["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
    elif case["op"] == "prefix":
        s["prefix_table"] = s["block_table"][0, :1].clone()
        s["prefix_len"] = torch.tensor([0], dtype=torch.int32, device="cuda")
    s["kv_lens"] = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([sum(q_len[:b]) for b in range(case["batch"] + 1)], dtype=torch.int32, device="cuda")
    s["q"] = torch.randn((sum(q_len), hq, d), generator=gen, device="cuda").to(dtype)
    s["max_q"], s["max_kv"] = max(q_len), max(kv_len)
    return s


# ------------------------------------------------------------ plain forms --


def _plain_extend(s):
    page = s["case"]["page"]
    new, kv = s["new_lens"].long(), s["kv_lens"].long()
    after = kv + new
    had, have = (kv + page - 1) // page, (after + page - 1) // page
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    taken = torch.cat([new.new_zeros(1), (have - had).cumsum(0)])
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    real = b < len(new)
    b = b.clamp(max=len(new) - 1)
    pos = torch.where(real, kv[b] + t - cu[b], 0)
    at = pos // page
    fresh = real & (at >= had[b])
    top = s["n_free"].long()
    free = s["free_pages"].long()[(top - 1 - (taken[b] + at - had[b])).clamp(min=0, max=len(s["free_pages"]) - 1)]
    paged = torch.where(fresh, free, s["block_table"].long()[b, at])
    slots = torch.where(real, paged * page + pos % page, -1)
    s["block_table"][b[fresh], at[fresh]] = paged[fresh].int()
    return after.int(), cu.int(), slots, pos, (top - taken[-1]).int(), s["block_table"]


def _plain_norm_rope(x, weight, s):
    c = s["case"]
    rot = c["rot"]
    x = x.float()
    if weight is not None:
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight.float()
    positions = s["positions"][s["axes"].long()].T if s["axes"] is not None else s["positions"].T
    angle = positions.double() * s["inv_freq"]   # far positions lose their angle in 32 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _values(rows):
    """Q8_0 rows -> float32 values."""
    blocks = rows.unflatten(-1, (-1, 34))
    scale = blocks[..., :2].contiguous().view(torch.float16).float()
    return (blocks[..., 2:].contiguous().view(torch.int8).float() * scale).flatten(-2)


def _plain_attention(s):
    c = s["case"]
    hk, d, page = c["kv_heads"], c["d"], c["page"]
    g, outs = c["heads"] // hk, []
    cu = s["cu_q"].long()
    n_q = cu[1:] - cu[:-1]
    key = torch.arange(s["block_table"].shape[1] * page, device="cuda")
    row = torch.arange(s["max_q"], device="cuda")
    # as many sequences at once as keep the scores and the values within some gigabytes
    step = max(1, (1 << 31) // (len(key) * max(c["heads"] * s["max_q"], 2 * hk * d)))
    for b0 in range(0, c["batch"], step):
        b1 = min(c["batch"], b0 + step)
        n, table, kv, nq = b1 - b0, s["block_table"][b0:b1].long(), s["kv_lens"][b0:b1].long()[:, None, None], n_q[b0:b1]
        k = _values(s["k_pages"][table].transpose(1, 2).reshape(n, hk, len(key), -1))
        v = _values(s["v_pages"][table].transpose(1, 2).reshape(n, hk, len(key), -1))
        at = (cu[b0:b1, None] + row).clamp(max=s["q"].shape[0] - 1)
        q = s["q"].float()[at].reshape(n, -1, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
        x = (q @ k.transpose(-1, -2) / math.sqrt(d)).view(n, hk, g, -1, len(key))
        p = kv - nq[:, None, None] + row[:, None]
        seen = (key <= p) & (key < kv)
        if c["op"] == "window":
            seen &= (key > p - c["window"]) | (key < c["sinks"])
        x = x.masked_fill_(~seen.view(n, 1, 1, -1, len(key)), -math.inf)
        top = x.amax(-1, keepdim=True)
        x = x.sub_(torch.where(top == -math.inf, 0, top)).exp_()
        total = x.sum(-1, keepdim=True)
        y = (x.view(n, hk, -1, len(key)) @ v).view(n, hk, g, -1, d) / torch.where(total == 0, 1, total)
        y = y.permute(0, 3, 1, 2, 4).reshape(n, -1, hk * g, d)
        outs.append(y[row < nq[:, None]].to(s["q"].dtype))
    return torch.cat(outs)


def run(s):
    c = s["case"]
    if own:
        from chunked_prefill_attention_gb300 import q8attn

        if c["op"] == "extend":
            kv, cu, slots, pos, n_free = q8attn.q8kv_extend_paged(s["new_lens"], s["kv_lens"], s["block_table"],
                                                                  s["free_pages"], s["n_free"], c["page"], s["total"])
            return kv, cu, slots, pos, n_free, s["block_table"]
        if c["op"] == "norm_rope":
            return q8attn.attn_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"],
                                         axes=s["axes"], eps=1e-6, interleaved=c["interleaved"])
        args = (s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["kv_lens"], s["cu_q"], s["max_q"], s["max_kv"])
        if c["op"] == "window":
            return q8attn.attn_paged_window(*args, c["window"], c["sinks"])
        return q8attn.attn_paged_prefix(*args, s["prefix_table"], s["prefix_len"])
    if c["op"] == "extend":
        return _plain_extend(s)
    if c["op"] == "norm_rope":
        return tuple(_plain_norm_rope(x, w, s).to(x.dtype) for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])))
    return _plain_attention(s)


def work(case):
    if case["op"] == "extend":
        n, page = case["batch"], case["page"]
        tokens = sum(_spread(case["max_new"], case["min_new"], n)) + case["padding"]
        return {"bytes": 16 * n + 16 * tokens + 8 * (tokens // page), "flops": 4 * tokens}
    d, size = case["d"], {_F16: 2, _BF16: 2, _F32: 4}[case["dtype"]]
    if case["op"] == "norm_rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * n * d * size + 8 * case["axes"] * case["tokens"],
                "flops": n * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    row = d // 32 * 34
    q, kv = _lengths(case)
    if case["op"] == "window":
        seen = [_visible(case, a, n) for a, n in zip(q, kv)]
        pairs, keys = sum(p for p, _ in seen), sum(k for _, k in seen)
    else:
        pairs = sum(a * n - a * (a - 1) // 2 for a, n in zip(q, kv))
        keys = case["prefix"] + sum(n - case["prefix"] for n in kv)
    return {"bytes": 2 * keys * case["kv_heads"] * row + 2 * sum(q) * case["heads"] * d * size,
            "flops": 4 * d * case["heads"] * pairs}


# -------------------------------------------------------- 64-bit definition --


def _exact_extend(case, s):
    """Sequence by sequence, on the host."""
    page = case["page"]
    new, kv, free = s["new_lens"].tolist(), s["kv_lens"].tolist(), s["free_pages"].tolist()
    table, left = s["block_table"].cpu().clone(), int(s["n_free"])
    cu, slots, positions = [0], [], []
    for b, (m, n) in enumerate(zip(new, kv)):
        while (n + page - 1) // page * page < n + m:   # pages one by one from the top of the stack
            left -= 1
            table[b, (n + page - 1) // page] = free[left]
            taken = min(m, (n + page - 1) // page * page + page - n)
            at = torch.arange(n, n + taken)
            slots.append(table[b, at // page].long() * page + at % page)
            positions.append(at)
            n, m = n + taken, m - taken
        at = torch.arange(n, n + m)
        slots.append(table[b, at // page].long() * page + at % page)
        positions.append(at)
        cu.append(cu[-1] + new[b])
        kv[b] = n + m
    pad = s["total"] - cu[-1]
    slots.append(torch.full((pad,), -1))
    positions.append(torch.zeros(pad, dtype=torch.int64))
    out = (torch.tensor(kv, dtype=torch.int32), torch.tensor(cu, dtype=torch.int32), torch.cat(slots),
           torch.cat(positions), torch.tensor([left], dtype=torch.int32), table)
    return tuple(t.cuda() for t in out)


def _exact_norm_rope(x, weight, case, s):
    """Each pair of channels as a complex number, turned by e^(i angle)."""
    y = x.double()
    if weight is not None:
        y = weight.double() * y / torch.sqrt(torch.einsum("thd,thd->th", y, y) / y.shape[-1] + 1e-6)[..., None]
    rot, h = case["rot"], case["rot"] // 2
    freq = torch.exp(-2 * torch.arange(h, dtype=torch.float64, device="cuda") / rot * math.log(10000.0))
    angle, first = [], 0
    for a, n in enumerate(_sections(h, case["axes"])):
        angle.append(torch.outer(s["positions"][a].double(), freq[first:first + n]))
        first += n
    angle = torch.cat(angle, 1)
    one = 2 * torch.arange(h, device="cuda") if case["interleaved"] else torch.arange(h, device="cuda")
    two = one + (1 if case["interleaved"] else h)
    y = y.clone()
    z = torch.complex(y[..., one], y[..., two]) * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_rows(pages, slots, d):
    """Rows by slot in 64 bits: [slots][kv_heads][d]."""
    rows = pages.permute(0, 2, 1, 3).reshape(-1, pages.shape[1], d // 32, 34)[slots]
    scale = rows[..., 0:2].contiguous().view(torch.float16).double()
    return (scale * rows[..., 2:34].contiguous().view(torch.int8).double()).reshape(len(slots), -1, d)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "extend":
        return _exact_extend(case, s)
    if case["op"] == "norm_rope":
        return tuple(_exact_norm_rope(s[x], s[x + "_weight"], case, s) for x in ("q", "k"))
    d, (q_len, kv_len) = case["d"], _lengths(case)
    if sum(a * n for a, n in zip(q_len, kv_len)) * case["heads"] > 1 << 34:
        return None   # minutes in 64 bits
    g, out, r0 = case["heads"] // case["kv_heads"], [], 0
    for b, (nq, n) in enumerate(zip(q_len, kv_len)):
        at = torch.arange(n, device="cuda")
        slots = s["block_table"][b].long()[at // case["page"]] * case["page"] + at % case["page"]
        q = s["q"][r0:r0 + nq].double()
        r0 += nq
        p = n - nq + torch.arange(nq, device="cuda")[:, None]
        hidden = at > p
        if case["op"] == "window":
            hidden |= (at <= p - case["window"]) & (at >= case["sinks"])
        y = torch.zeros_like(q)
        for kh in range(case["kv_heads"]):
            k = _exact_rows(s["k_pages"][:, kh:kh + 1], slots, d)[:, 0]
            v = _exact_rows(s["v_pages"][:, kh:kh + 1], slots, d)[:, 0]
            for h in range(kh * g, (kh + 1) * g):
                a = torch.einsum("id,jd->ij", q[:, h], k) * d ** -0.5
                y[:, h] = torch.softmax(torch.where(hidden, torch.full_like(a, -math.inf), a), dim=1) @ v
        out.append(y)
    return torch.cat(out)
