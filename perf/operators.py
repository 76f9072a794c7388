"""The paged Q8_0 cache and the attention over it, as a server runs them, with plain forms of the same operators.

Q8_0 rows: a head row of D channels is D / 32 blocks of 34 bytes, an fp16 scale d and 32 int8 codes c; its values are
d * c.  Pages: uint8 [n_pages][kv_heads][page_tokens][D / 32 * 34]; a row's slot is page * page_tokens + offset.
"""

import math

import torch

own = False

_F16, _BF16, _F32 = "float16", "bfloat16", "float32"


def listed():
    return [
        # rotation of the queries of one step of a batch of 64 sequences
        {"name": "rope_step", "op": "rope", "tokens": 64, "heads": 32, "d": 64, "rot": 64, "interleaved": False,
         "dtype": _F16, "factor": 1.0, "max_pos": 65536, "packed": False},
        # the queries of a 16,384-token prompt, a slice of the fused projection's output, half of each head rotated,
        # positions stretched eightfold for a long context
        {"name": "rope_prompt", "op": "rope", "tokens": 16384, "heads": 32, "d": 128, "rot": 64, "interleaved": True,
         "dtype": _BF16, "factor": 8.0, "max_pos": 1048576, "packed": True},
        # the new keys and values of one step of 64 sequences, written and read back
        {"name": "append_step", "op": "append", "tokens": 64, "heads": 8, "d": 128, "page": 16, "rot": 128,
         "interleaved": False, "dtype": _BF16, "factor": 1.0, "max_pos": 65536, "pages": 1024, "packed": False},
        # the keys and values of a 16,384-token prompt
        {"name": "append_prompt", "op": "append", "tokens": 16384, "heads": 32, "d": 64, "page": 64, "rot": 64,
         "interleaved": True, "dtype": _F16, "factor": 8.0, "max_pos": 1048576, "pages": 320, "packed": True},
        # a prefix of 2,047 tokens handed to another consumer in bf16
        {"name": "read_prefix", "op": "read", "tokens": 2047, "heads": 8, "d": 128, "page": 16, "dtype": _BF16,
         "pages": 512},
        # a whole 262,144-token context read back
        {"name": "read_context", "op": "read", "tokens": 262144, "heads": 8, "d": 64, "page": 128, "dtype": _F16,
         "pages": 2048},
        # one new token after a short context: latency
        {"name": "decode_one", "op": "attn", "batch": 1, "max_q": 1, "min_q": 1, "max_kv": 511, "min_kv": 511,
         "heads": 32, "kv_heads": 8, "d": 64, "page": 16, "dtype": _F16, "causal": True},
        # one new token for each of 64 sequences of very different lengths
        {"name": "decode_batch", "op": "attn", "batch": 64, "max_q": 1, "min_q": 1, "max_kv": 16384, "min_kv": 300,
         "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "dtype": _BF16, "causal": True},
        # one new token after a million, a key and value head for every query head
        {"name": "decode_long", "op": "attn", "batch": 1, "max_q": 1, "min_q": 1, "max_kv": 1048575,
         "min_kv": 1048575, "heads": 32, "kv_heads": 32, "d": 64, "page": 128, "dtype": _F16, "causal": True},
        # bursts of 16 candidate tokens for each of four sequences
        {"name": "verify_burst", "op": "attn", "batch": 4, "max_q": 16, "min_q": 9, "max_kv": 32768, "min_kv": 9000,
         "heads": 32, "kv_heads": 8, "d": 64, "page": 32, "dtype": _F16, "causal": True},
        # chunks of new tokens after long contexts
        {"name": "prompt_chunk", "op": "attn", "batch": 3, "max_q": 2048, "min_q": 700, "max_kv": 32768,
         "min_kv": 12000, "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "dtype": _BF16, "causal": True},
        # whole prompts of different lengths in one call
        {"name": "prompt_whole", "op": "attn", "batch": 4, "max_q": 8192, "min_q": 1501, "max_kv": 0, "min_kv": 0,
         "heads": 32, "kv_heads": 32, "d": 64, "page": 128, "dtype": _F16, "causal": True},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    d = rng.choice([64, 128])
    dtype = rng.choice([_F16, _BF16])
    page = rng.choice([16, 32, 64, 128, 256])
    rotary = {"rot": rng.choice([d, d // 2, d // 4]), "interleaved": rng.random() < 0.5,
              "factor": rng.choice([1.0, 4.0, 8.0]), "max_pos": log_int(1000, 1 << 20), "packed": rng.random() < 0.5}
    op = rng.choice(["rope", "append", "read", "attn", "attn", "attn"])
    if op == "rope":
        return {"op": op, "tokens": log_int(1, 16384), "heads": rng.choice([1, 5, 8, 24, 32]), "d": d,
                "dtype": rng.choice([_F16, _BF16, _F32]), **rotary}
    if op == "append":
        tokens = log_int(1, 16384)
        return {"op": op, "tokens": tokens, "heads": rng.choice([1, 3, 8, 16]), "d": d, "page": page,
                "dtype": rng.choice([_F16, _BF16, _F32]), "pages": -(-tokens // page) + log_int(1, 200), **rotary}
    if op == "read":
        tokens = log_int(1, 131072)
        return {"op": op, "tokens": tokens, "heads": rng.choice([1, 3, 8]), "d": d, "page": page, "dtype": dtype,
                "pages": -(-tokens // page) + log_int(1, 200)}
    kv_heads = rng.choice([1, 2, 8])
    case = {"op": op, "heads": kv_heads * rng.choice([1, 3, 4, 8]), "kv_heads": kv_heads, "d": d, "page": page,
            "dtype": dtype, "causal": rng.random() < 0.8}
    kind = rng.choice(["decode", "burst", "chunk", "whole"])
    if kind == "decode":
        batch = log_int(1, 64)
        hi = log_int(20, min(262144, 2097152 // batch))
        return {**case, "batch": batch, "max_q": 1, "min_q": 1, "max_kv": hi, "min_kv": max(1, hi // 9)}
    if kind == "burst":
        batch, q = log_int(1, 8), rng.randint(2, 64)
        hi = log_int(100, 65536)
        return {**case, "batch": batch, "max_q": q, "min_q": max(1, q // 2), "max_kv": hi, "min_kv": max(q, hi // 5)}
    if kind == "chunk":
        batch, q = rng.randint(1, 4), log_int(65, 2048)
        hi = q + log_int(50, 16384)
        return {**case, "batch": batch, "max_q": q, "min_q": max(1, q // 6), "max_kv": hi, "min_kv": q}
    batch, q = rng.randint(1, 4), log_int(30, 5000)
    return {**case, "batch": batch, "max_q": q, "min_q": max(1, q // 4), "max_kv": 0, "min_kv": 0}


# ---------------------------------------------------------------- inputs --


def _lengths(case):
    """(new tokens, keys) of each sequence: between the case's bounds, the first at the largest, odd ones among them."""
    n = case["batch"]
    q = [case["max_q"] - (case["max_q"] - case["min_q"]) * ((5 * i) % n) // max(1, n - 1) for i in range(n)]
    kv = [max(case["max_kv"] - (case["max_kv"] - case["min_kv"]) * i // max(1, n - 1), a) for i, a in enumerate(q)]
    return q, kv


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = getattr(torch, case["dtype"])
    d, s = case["d"], {"case": dict(case)}
    if case["op"] in ("rope", "append"):
        n, h = case["tokens"], case["heads"]
        rot = case["rot"]
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot) / case["factor"]
        start = torch.randint(0, max(1, case["max_pos"] - n), (1,), generator=gen, device="cuda")
        s["positions"] = start + torch.arange(n, device="cuda")
        if n <= 256:   # a step: each token its own sequence's position
            s["positions"] = torch.randint(0, case["max_pos"], (n,), generator=gen, device="cuda")
        # the projections' output: the tensors are slices of one buffer, or each has its own
        make = lambda: torch.randn((n, h * (3 if case["packed"] else 1), d), generator=gen, device="cuda").to(dtype)
        if case["op"] == "rope":
            s["x"] = make()[:, :h]
            return s
        if case["packed"]:
            _, s["k"], s["v"] = make().split(h, dim=1)
        else:
            s["k"], s["v"] = make(), make()
    if case["op"] in ("append", "read"):
        page, n_pages = case["page"], case["pages"]
        s["k_pages"] = _random_pages(n_pages, case["heads"], page, d, gen)
        s["v_pages"] = _random_pages(n_pages, case["heads"], page, d, gen)
        order = torch.randperm(n_pages, generator=gen, device="cuda")
        at = torch.arange(case["tokens"], device="cuda")
        s["slots"] = order[at // page] * page + at % page
        if case["tokens"] <= 256:   # a step: rows of different sequences
            s["slots"] = torch.randperm(n_pages * page, generator=gen, device="cuda")[:case["tokens"]]
        return s
    q_len, kv_len = _lengths(case)
    page, width = case["page"], -(-max(kv_len) // case["page"])
    used = [-(-n // page) for n in kv_len]
    n_pages = sum(used) + 1
    s["k_pages"] = _random_pages(n_pages, case["kv_heads"], page, d, gen)
    s["v_pages"] = _random_pages(n_pages, case["kv_heads"], page, d, gen)
    order = torch.randperm(n_pages, generator=gen, device="cuda").int()
    s["block_table"] = torch.zeros((case["batch"], width), dtype=torch.int32, device="cuda")
    first = 0
    for b, n in enumerate(used):
        s["block_table"][b, :n] = order[first:first + n]
        first += n
    s["kv_lens"] = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([sum(q_len[:b]) for b in range(case["batch"] + 1)], dtype=torch.int32, device="cuda")
    s["q"] = torch.randn((sum(q_len), case["heads"], d), generator=gen, device="cuda").to(dtype)
    s["max_q"], s["max_kv"] = max(q_len), max(kv_len)
    return s


# ------------------------------------------------------------ plain forms --


def _rotate(x, s):
    """Rotary positions in 64 bits: channel pairs (i, i + rot / 2), or (2i, 2i + 1) in the interleaved layout."""
    rot = s["case"]["rot"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    x = x.double()
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _quantise(x):
    """float64 [..., D] -> Q8_0 rows, uint8 [..., D / 32 * 34]."""
    x = x.unflatten(-1, (-1, 32))
    scale = (x.abs().amax(-1, keepdim=True) / 127).float().half()
    y = x / torch.where(scale == 0, 1, scale).double()
    codes = (y.sign() * (y.abs() + 0.5).floor()).clamp(-127, 127)
    codes = torch.where(scale == 0, 0, codes).to(torch.int8)
    return torch.cat([scale.view(torch.uint8), codes.view(torch.uint8)], -1).flatten(-2)


def _values(rows):
    """Q8_0 rows -> float32 values."""
    blocks = rows.unflatten(-1, (-1, 34))
    scale = blocks[..., :2].contiguous().view(torch.float16).float()
    return (blocks[..., 2:].contiguous().view(torch.int8).float() * scale).flatten(-2)


def _plain_attention(s):
    c = s["case"]
    b, hk, d, page = c["batch"], c["kv_heads"], c["d"], c["page"]
    g, mq = c["heads"] // hk, s["max_q"]
    table = s["block_table"].long()
    keys = table.shape[1] * page
    k = _values(s["k_pages"][table].transpose(1, 2).reshape(b, hk, keys, -1))
    v = _values(s["v_pages"][table].transpose(1, 2).reshape(b, hk, keys, -1))
    n_q = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    row = torch.arange(mq, device="cuda")
    at = (s["cu_q"][:-1, None].long() + row).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[at].reshape(b, mq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * mq, d)
    x = (q @ k.transpose(-1, -2) / math.sqrt(d)).view(b, hk, g, mq, keys)
    kv = s["kv_lens"].long()[:, None, None]
    key = torch.arange(keys, device="cuda")
    seen = (key < kv) & ((key <= kv - n_q[:, None, None] + row[:, None]) if c["causal"] else key >= 0)
    x = x.masked_fill_(~seen.view(b, 1, 1, -1, keys), -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    y = (x.view(b, hk, g * mq, keys) @ v).view(b, hk, g, mq, d) / torch.where(total == 0, 1, total)
    y = y.permute(0, 3, 1, 2, 4).reshape(b, mq, hk * g, d)
    return y[row < n_q[:, None]].to(s["q"].dtype)


def run(s):
    c = s["case"]
    if own:
        from chunked_prefill_attention_gb300 import q8attn

        if c["op"] == "rope":
            return q8attn.attn_rope(s["x"], s["positions"], s["inv_freq"], interleaved=c["interleaved"])
        if c["op"] == "append":
            q8attn.q8kv_append_paged(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slots"], s["positions"],
                                     s["inv_freq"], interleaved=c["interleaved"])
            return q8attn.q8kv_read_paged(s["k_pages"], s["v_pages"], s["slots"], torch.float16)
        if c["op"] == "read":
            return q8attn.q8kv_read_paged(s["k_pages"], s["v_pages"], s["slots"], getattr(torch, c["dtype"]))
        return q8attn.attn_paged(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["kv_lens"], s["cu_q"],
                                 s["max_q"], s["max_kv"], causal=c["causal"])
    if c["op"] == "rope":
        return _rotate(s["x"], s).to(s["x"].dtype)
    if c["op"] == "attn":
        return _plain_attention(s)
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    if c["op"] == "append":
        s["k_pages"][page, :, off] = _quantise(_rotate(s["k"], s))
        s["v_pages"][page, :, off] = _quantise(s["v"].double())
    dtype = torch.float16 if c["op"] == "append" else getattr(torch, c["dtype"])
    return _values(s["k_pages"][page, :, off]).to(dtype), _values(s["v_pages"][page, :, off]).to(dtype)


def work(case):
    d, size = case["d"], {_F16: 2, _BF16: 2, _F32: 4}[case["dtype"]]
    row = d // 32 * 34
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * d * size + 8 * case["tokens"], "flops": 3 * n * case["rot"]}
    if case["op"] == "append":   # inputs read, rows written, rows read back, values written
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * (d * size + row + row + 2 * d) + 24 * case["tokens"], "flops": 10 * n * d}
    if case["op"] == "read":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * (row + d * size) + 8 * case["tokens"], "flops": 2 * n * d}
    q, kv = _lengths(case)
    pairs = sum(a * n - (a * (a - 1) // 2 if case["causal"] else 0) for a, n in zip(q, kv))
    moved = 2 * sum(kv) * case["kv_heads"] * row + 2 * sum(q) * case["heads"] * d * size
    return {"bytes": moved, "flops": 4 * d * case["heads"] * pairs}


# -------------------------------------------------------- 64-bit definition --


def _exact_rotation(x, case, positions):
    """Each pair of channels as a complex number, turned by e^(i angle)."""
    rot, h = case["rot"], case["rot"] // 2
    i = torch.arange(h, dtype=torch.float64, device="cuda")
    angle = torch.outer(positions.double(), torch.exp(-2 * i / rot * math.log(10000.0)) / case["factor"])
    first = 2 * torch.arange(h, device="cuda") if case["interleaved"] else torch.arange(h, device="cuda")
    second = first + (1 if case["interleaved"] else h)
    y = x.double()
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_dequantised(x):
    """What Q8_0 holds of float64 values x, in 64 bits."""
    y = x.reshape(-1, 32)
    scale = (y.abs().max(dim=1, keepdim=True).values / 127).to(torch.float32).to(torch.float16).double()
    t = torch.where(scale > 0, y / scale, torch.zeros_like(y))
    c = torch.minimum(torch.floor(t.abs() + 0.5), torch.full_like(t, 127.0)) * torch.sign(t)
    return (c * scale).reshape(x.shape)


def _exact_rows(pages, slots, d):
    """Rows by slot in 64 bits: [slots][kv_heads][d]."""
    rows = pages.permute(0, 2, 1, 3).reshape(-1, pages.shape[1], d // 32, 34)[slots]
    scale = rows[..., 0:2].contiguous().view(torch.float16).double()
    return (scale * rows[..., 2:34].contiguous().view(torch.int8).double()).reshape(len(slots), -1, d)


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "rope":
        return _exact_rotation(s["x"], case, s["positions"])
    if case["op"] == "append":
        return _exact_dequantised(_exact_rotation(s["k"], case, s["positions"])), _exact_dequantised(s["v"].double())
    if case["op"] == "read":
        return _exact_rows(s["k_pages"], s["slots"], d), _exact_rows(s["v_pages"], s["slots"], d)
    q_len, kv_len = _lengths(case)
    g, out, r0 = case["heads"] // case["kv_heads"], [], 0
    for b, (nq, n) in enumerate(zip(q_len, kv_len)):
        at = torch.arange(n, device="cuda")
        slots = s["block_table"][b].long()[at // case["page"]] * case["page"] + at % case["page"]
        q = s["q"][r0:r0 + nq].double()
        r0 += nq
        last = n - nq + torch.arange(nq, device="cuda") if case["causal"] else torch.full((nq,), n, device="cuda")
        y = torch.zeros_like(q)
        for kh in range(case["kv_heads"]):
            k = _exact_rows(s["k_pages"][:, kh:kh + 1], slots, d)[:, 0]
            v = _exact_rows(s["v_pages"][:, kh:kh + 1], slots, d)[:, 0]
            for h in range(kh * g, (kh + 1) * g):
                a = torch.einsum("id,jd->ij", q[:, h], k) * d ** -0.5
                a = torch.where(at[None, :] > last[:, None], torch.full_like(a, -math.inf), a)
                w = torch.softmax(a, dim=1)
                y[:, h] = w @ v
        out.append(y)
    return torch.cat(out)
