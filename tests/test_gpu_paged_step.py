"""The tables of a step and the norms with rotary positions, against plain implementations.

Tolerances of attn_norm_rope.  An output is rounded once to its type: u = finfo.eps / 2 of its value.  The mean of D <= 128
squares in fp32: every square and every addition is off by 2^-24 of the (positive) sum, at most 24 of them one after
another, so 2^-19 of it; its root half of that; rsqrtf 2 units, 2^-22; two products 2^-23: 2^-19 of the normalised value
bounds all.  The rotation adds 2^-22 (|a| + |b|) and 2^-51 of the angle (products and sums in fp32, angles, sincospif).
"""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def Q(lib):
    from chunked_prefill_attention_gb300 import q8attn
    yield q8attn
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def clean_status(Q):
    yield
    rc, word = Q.device_status(clear=True)
    assert rc == 0, hex(word)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ tables --


def extend(new, kv, table, free, n_free, page, total):
    """Sequence by sequence, as the definition reads; also whether anything was refused."""
    table, kv, wrong = table.clone(), list(kv), False
    cu, slots, pos = [0], [-1] * total, [0] * total
    left = n_free
    wanted = 0   # pages of all sequences so far, the refused ones' too
    for b, n in enumerate(new):
        rows = max(n, 0)
        r0 = cu[-1]
        cu.append(r0 + rows)
        valid = n >= 0 and kv[b] >= 0 and kv[b] + n <= table.shape[1] * page
        need = -(-(kv[b] + n) // page) - -(-kv[b] // page) if valid else 0
        wanted += need
        if not valid or (need and wanted > n_free) or (rows and cu[-1] > total):
            wrong = True
            continue
        first = -(-kv[b] // page)
        for i in range(need):
            left -= 1
            table[b, first + i] = free[left]
        for i in range(n):
            p = kv[b] + i
            slots[r0 + i], pos[r0 + i] = int(table[b, p // page]) * page + p % page, p
        kv[b] += n
    return kv, [min(c, total) for c in cu], slots, pos, left, table, wrong


EXTEND = [
    # sequences, most new tokens, most keys before, page, rows of padding
    (1, 1, 0, 16, 0), (1, 1, 1, 16, 3), (1, 40, 100, 16, 0), (3, 5, 200, 64, 1), (64, 1, 5000, 64, 0), (33, 17, 900, 16, 31),
    (1000, 1, 300, 32, 7), (1025, 4, 60, 16, 0), (7, 3000, 0, 128, 100), (2, 5001, 77, 4096, 0), (2500, 9, 40, 16, 900),
]


def build(case, seed):
    batch, most_new, most_kv, page, padding = case
    g = gen(seed)
    new = torch.randint(0, most_new + 1, (batch,), generator=g, device="cuda").int()
    kv = torch.randint(0, most_kv + 1, (batch,), generator=g, device="cuda").int()
    new[0], kv[-1] = most_new, most_kv
    had = -(-kv // page)
    lack = int((-(-(kv + new) // page) - had).sum())
    order = torch.randperm(int(had.sum()) + lack + 5, generator=g, device="cuda").int()
    width = -(-(most_new + most_kv) // page) + 1
    table = torch.full((batch, width), -7, dtype=torch.int32, device="cuda")
    first = 0
    for b, n in enumerate(had.tolist()):
        table[b, :n] = order[first:first + n]
        first += n
    return new, kv, table, order[first:].contiguous(), lack, page, int(new.sum()) + padding


def same(got, table, want):
    for x, y in zip((*got, table), want):
        assert torch.equal(x.cpu().flatten(), torch.as_tensor(y).flatten().to(x.dtype)), (x, y)


@pytest.mark.parametrize("case", EXTEND)
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(Q, case, in_place):
    new, kv, table, free, lack, page, total = build(case, 1)
    n_free = torch.tensor([len(free)], dtype=torch.int32, device="cuda")
    *want, wrong = extend(new.tolist(), kv.tolist(), table.cpu(), free.cpu(), len(free), page, total)
    assert not wrong
    out = None
    if in_place:
        long = lambda n: torch.full((n,), -99, dtype=torch.int64, device="cuda")
        out = kv, torch.full((len(new) + 1,), -99, dtype=torch.int32, device="cuda"), long(total), long(total), n_free
    before = free.clone(), kv.clone()
    got = Q.q8kv_extend_paged(new, kv, table, free, n_free, page, total, out=out)
    same(got, table, want)
    assert torch.equal(free, before[0])
    assert (got[0].data_ptr() == kv.data_ptr()) == in_place and (in_place or torch.equal(kv, before[1]))


@pytest.mark.parametrize("case", EXTEND[2:])
@pytest.mark.parametrize("fault", ["pages", "rows", "table", "negative", "all"])
def test_extend_leaves_what_it_cannot_serve(Q, case, fault):
    """Sequences that lack pages, room in the table or rows, or with negative lengths stay as they are; the others are
    served, and the failure is recorded."""
    new, kv, table, free, lack, page, total = build(case, 2)
    left = len(free)
    if fault in ("pages", "all"):
        left = lack // 2
    if fault in ("rows", "all"):
        total = int(new.sum()) * 2 // 3
    if fault in ("table", "all"):
        kv[len(kv) // 3] = table.shape[1] * page
        new[len(kv) // 3] = 1
        if fault == "table":
            total = int(new.sum())
    if fault in ("negative", "all"):
        new[len(new) // 2] = -3
        kv[-1] = -1
        total = int(new.clamp(min=0).sum()) - (total if fault == "all" else 0) % 2
    *want, wrong = extend(new.tolist(), kv.tolist(), table.cpu(), free.cpu(), left, page, total)
    n_free = torch.tensor([left], dtype=torch.int32, device="cuda")
    got = Q.q8kv_extend_paged(new, kv, table, free, n_free, page, total)
    same(got, table, want)
    rc, word = Q.device_status(clear=True)
    assert (rc != 0) == wrong


def test_extend_bad_pages_and_counts(Q):
    """Page numbers below 0 and more free pages than the list holds are recorded and not followed."""
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = torch.tensor([[3, -1], [-5, 0]], dtype=torch.int32, device="cuda")
    kv, cu, slots, pos, left = Q.q8kv_extend_paged(i32(2, 1), i32(15, 3), table, i32(-2, 9), i32(2), 16, 4)
    assert slots.tolist() == [63, 144, -1, -1] and pos.tolist() == [15, 16, 3, 0] and left.tolist() == [1]
    assert table.tolist() == [[3, 9], [-5, 0]]
    assert Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG
    kv, cu, slots, pos, left = Q.q8kv_extend_paged(i32(1), i32(16), table[:1], i32(4, 6), i32(50), 16, 1)
    assert slots.tolist() == [96] and left.tolist() == [1]
    assert Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG
    kv, cu, slots, pos, left = Q.q8kv_extend_paged(i32(1), i32(16), table[:1], i32(4, 6), i32(-1), 16, 1)
    assert slots.tolist() == [-1] and kv.tolist() == [16] and left.tolist() == [0]
    assert Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG


def test_extend_nothing(Q):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    for total in (0, 5, 5000):
        n_free = torch.tensor([0], dtype=torch.int32, device="cuda")
        kv, cu, slots, pos, left = Q.q8kv_extend_paged(none, none, table, none, n_free, 16, total)
        assert cu.tolist() == [0] and left.tolist() == [0] and (slots == -1).all() and (pos == 0).all()


@pytest.mark.parametrize("batch,new_tokens", [(50, 1), (40, 300)])
def test_extend_captured(Q, batch, new_tokens):
    """A captured step in place goes on by itself; new_lens may change between replays."""
    page, steps = 16, 5
    kv = torch.arange(batch, dtype=torch.int32, device="cuda")
    had = -(-kv // page)
    width = (batch + steps * new_tokens) // page + 2
    n_pages = batch * width
    order = torch.randperm(n_pages, generator=gen(4), device="cuda").int()
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    first = 0
    for b, n in enumerate(had.tolist()):
        table[b, :n] = order[first:first + n]
        first += n
    free = order[first:].contiguous()
    n_free = torch.tensor([len(free)], dtype=torch.int32, device="cuda")
    new = torch.full((batch,), new_tokens, dtype=torch.int32, device="cuda")
    total = batch * new_tokens
    out = (kv, torch.empty(batch + 1, dtype=torch.int32, device="cuda"), torch.empty(total, dtype=torch.int64, device="cuda"),
           torch.empty(total, dtype=torch.int64, device="cuda"), n_free)
    state = [new.tolist(), kv.tolist(), table.cpu(), free.cpu(), len(free)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.q8kv_extend_paged(new, kv, table, free, n_free, page, total, out=out)
    for step in range(steps):
        if step == 3:
            new[::3] = 0
            state[0] = new.tolist()
        graph.replay()
        *want, wrong = extend(*state, page, total)
        assert not wrong
        same(out, table, want)
        state[1], state[4], state[2] = want[0], want[4], want[5]


def test_extend_refusals(Q):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    good = lambda: dict(new_lens=i32(1, 1), kv_lens=i32(0, 0), block_table=torch.zeros((2, 2), dtype=torch.int32, device="cuda"),
                        free_pages=i32(1, 2, 3), n_free=i32(3), page_tokens=16, total_q=2)
    Q.q8kv_extend_paged(**good())
    for kw in (dict(new_lens=i32(1)), dict(kv_lens=i32(0, 0).long()), dict(kv_lens=i32(0, 0).cpu()), dict(n_free=i32(1, 1)),
               dict(block_table=torch.zeros((3, 2), dtype=torch.int32, device="cuda")), dict(total_q=-1),
               dict(block_table=torch.zeros((2, 4), dtype=torch.int32, device="cuda")[:, ::2]), dict(page_tokens=20),
               dict(free_pages=None), dict(new_lens=i32(1, 1, 1, 1)[::2])):
        with pytest.raises(Q.Q8AttnError):
            Q.q8kv_extend_paged(**{**good(), **kw})


# -------------------------------------------------------------- norm, rope --


def norm_rope64(x, weight, positions, inv_freq, axes, eps, interleaved, mscale=1.0):
    """The formula in 64 bits (CPU), and the bound of its fp32 evaluation."""
    x = x.double().cpu()
    bound = torch.zeros_like(x)
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double().cpu()
        bound = 2.0 ** -19 * x.abs()
    if inv_freq is None:
        return x, bound
    rot = 2 * len(inv_freq)
    positions = positions.cpu().double().reshape(-1, x.shape[0])
    axes = torch.zeros(rot // 2, dtype=torch.long) if axes is None else axes.cpu().long()
    angle = positions[axes].T * inv_freq.cpu()
    c, s = angle.cos()[:, None] * mscale, angle.sin()[:, None] * mscale
    first = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    second = first + (1 if interleaved else rot // 2)
    a, b = x[..., first], x[..., second]
    y = x.clone()
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    e = ((2.0 ** -22 + 2.0 ** -51 * angle.abs()[:, None]) * (a.abs() + b.abs()) + bound[..., first] + bound[..., second]) * abs(mscale)
    bound[..., first] = bound[..., second] = e
    return y, bound


def near(got, want, bound):
    u = torch.finfo(got.dtype).eps / 2
    got = got.double().cpu()
    ok = (got - want).abs() <= bound + u * (want.abs() + bound) + 2.0 ** -25
    assert ok.all(), (int((~ok).sum()), float((got - want).abs().max()))


NORM = [
    # tokens, heads, kv heads, D, rot, axes, interleaved, type, weights' type, largest position
    (1, 1, 0, 64, 64, 1, False, F16, F16, 10),
    (1, 32, 8, 128, 128, 1, False, BF16, BF16, 1 << 20),
    (64, 32, 8, 128, 128, 1, False, BF16, F32, 1 << 20),
    (7, 5, 1, 128, 128, 3, True, BF16, BF16, 5000),
    (33, 3, 3, 64, 64, 2, False, F32, F32, 1 << 31),
    (9, 4, 2, 64, 32, 1, True, F16, F16, 1 << 17),
    (130, 24, 24, 64, 64, 3, True, F16, F16, 4096),
    (9, 2, 1, 64, 24, 2, False, BF16, F16, 5000),      # rot / 2 not a multiple of the 16-byte access
    (9, 2, 2, 128, 10, 1, True, F16, BF16, 5000),
    (5, 1, 1, 128, 2, 1, False, F32, F32, 100),
    (1030, 3, 1, 128, 64, 1, False, F16, F16, 1 << 20),
    (2051, 1, 1, 64, 48, 3, True, F32, BF16, 1 << 16),
    (300, 40, 10, 128, 96, 4, False, BF16, BF16, 1 << 16),
    (515, 17, 3, 128, 128, 1, True, F32, F32, 1 << 16),
    (77, 7, 5, 64, 16, 1, False, F16, F16, 1 << 16),
]


def inputs(Q, case, seed, form):
    tokens, heads, kv, D, rot, n_axes, inter, dtype, w_type, far = case
    g = gen(seed)
    wide = (torch.randn((tokens, heads + 2 * kv + 1, D), generator=g, device="cuda") * 2).to(dtype)
    q, k = wide[:, :heads], wide[:, heads:heads + kv]
    if form in ("fresh", "odd offset"):
        apart = []
        for x in (q, k):
            flat = torch.empty(x.numel() + 1, dtype=dtype, device="cuda")
            at = 1 if form == "odd offset" else 0
            apart.append(flat[at:at + x.numel()].view(x.shape).copy_(x))
        q, k = apart
    pos = torch.randint(-far, far, (n_axes, tokens), generator=g, device="cuda")
    f = Q.rope_inv_freq(rot, factor=1.5, device="cuda")
    axes = torch.randint(0, n_axes, (rot // 2,), generator=g, device="cuda").int() if n_axes > 1 else None
    w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(w_type) for _ in range(2)]
    return wide, q, (k if kv else None), w[0], (w[1] if kv else None), pos, f, axes


@pytest.mark.parametrize("case", NORM)
@pytest.mark.parametrize("form", ["fresh", "slice", "in place", "odd offset"])
def test_norm_rope(Q, case, form):
    tokens, heads, kv, D, rot, n_axes, inter, dtype, w_type, far = case
    wide, q, k, qw, kw, pos, f, axes = inputs(Q, case, 1, form)
    want = [norm_rope64(x, w, pos, f, axes, 1e-5, inter, 0.75) for x, w in ((q, qw), (k, kw)) if x is not None]
    before = wide.clone()
    got = Q.attn_norm_rope(q, k, qw, kw, pos if n_axes > 1 else pos[0], f, axes=axes, eps=1e-5, interleaved=inter, mscale=0.75,
                           out=(q, k) if form == "in place" else None)
    for y, (w, b) in zip(got, want):
        near(y, w, b)
    if form == "in place":
        assert torch.equal(wide[:, heads + kv:], before[:, heads + kv:])
    else:
        assert torch.equal(wide, before)


@pytest.mark.parametrize("case", NORM[::3])
@pytest.mark.parametrize("what", ["turn only", "norm only", "q's norm only"])
def test_norm_rope_parts(Q, case, what):
    tokens, heads, kv, D, rot, n_axes, inter, dtype, w_type, far = case
    wide, q, k, qw, kw, pos, f, axes = inputs(Q, case, 2, "slice")
    if what == "turn only":
        qw = kw = None
    elif what == "norm only":
        pos = f = axes = None
    else:
        kw = None
    got = Q.attn_norm_rope(q, k, qw, kw, pos, f, axes=axes, interleaved=inter)
    for y, x, w in ((got[0], q, qw), (got[1], k, kw)):
        if x is not None:
            near(y, *norm_rope64(x, w, pos, f, axes, 1e-6, inter))
    if what == "turn only" and n_axes == 1:   # what attn_rope computes, to the bit
        assert torch.equal(got[0], Q.attn_rope(q, pos[0], f, interleaved=inter))


def test_norm_rope_extremes(Q):
    """Rows of zeros, the smallest and the largest values, infinities and NaN, with and without eps: each row by itself."""
    q = torch.zeros((6, 2, 64), dtype=F32, device="cuda")
    q[1, 0] = 2.0 ** -60
    q[2, 1] = 2.0 ** 55
    q[3, 0, 5] = float("inf")
    q[4, 1, 7] = float("nan")
    q[5, 1, 9] = 1.0
    w = torch.ones(64, device="cuda")
    y, _ = Q.attn_norm_rope(q, None, w, eps=1e-6)
    assert (y[0] == 0).all() and torch.allclose(y[1, 0], torch.full((64,), 2.0 ** -60 * 1000, device="cuda"))
    assert torch.allclose(y[2, 1], w) and (y[2, 0] == 0).all()
    assert y[3, 0, 5].isnan() and (y[3, 0, :5] == 0).all() and (y[3, 1] == 0).all()
    assert y[4, 1].isnan().all() and (y[4, 0] == 0).all()
    assert abs(y[5, 1, 9].item() - 8) < 1e-3
    y, _ = Q.attn_norm_rope(q, None, w, eps=0.0)
    assert y[0].isnan().all() and torch.allclose(y[1, 0], w)   # 0 / 0 is the formula's


def test_norm_rope_far_apart_tokens(Q):
    """Tokens more than 2^31 elements apart, and an empty call."""
    stride = (1 << 30) + 64
    flat = torch.empty(3 * stride, dtype=F16, device="cuda")
    q = flat.as_strided((3, 2, 64), (stride, 64, 1))
    q.copy_(torch.randn((3, 2, 64), generator=gen(3), device="cuda"))
    w = torch.ones(64, dtype=F16, device="cuda")
    pos, f = torch.tensor([5, 1 << 40, -3], device="cuda"), Q.rope_inv_freq(64, device="cuda")
    want, bound = norm_rope64(q, w, pos, f, None, 1e-6, False)
    got, _ = Q.attn_norm_rope(q, None, w, None, pos, f)
    near(got, want, bound)
    Q.attn_norm_rope(q, None, w, None, pos, f, out=(q, None))
    assert torch.equal(got, q)
    del flat, q
    torch.cuda.empty_cache()
    none = torch.empty((0, 2, 64), dtype=F16, device="cuda")
    y, _ = Q.attn_norm_rope(none, None, w, None, pos[:0], f)
    assert y.shape == none.shape


@pytest.mark.parametrize("odd", [False, True])
def test_norm_rope_most_heads(Q, odd):
    """The most heads of queries and keys that the call takes, one token."""
    D, n = 64, 65535
    flat = torch.randn(2 * n * D + 1, generator=gen(9), device="cuda").half()
    flat = flat[1:] if odd else flat[:-1]
    q, k = flat[:n * D].view(1, n, D), flat[n * D:].view(1, n, D)
    pos, f, w = torch.tensor([77], device="cuda"), Q.rope_inv_freq(D, device="cuda"), torch.ones(D, device="cuda")
    got = Q.attn_norm_rope(q, k, w, w, pos, f)
    for y, x in zip(got, (q, k)):
        near(y, *norm_rope64(x, w, pos, f, None, 1e-6, False))


def test_norm_rope_bad_axis(Q):
    """An axis that does not exist is recorded and taken for axis 0."""
    q = torch.randn((2, 1, 64), generator=gen(6), device="cuda")
    pos = torch.tensor([[1, 2], [30, 40]], device="cuda")
    f = Q.rope_inv_freq(64, device="cuda")
    axes = torch.ones(32, dtype=torch.int32, device="cuda")
    axes[3], axes[9] = 2, -1
    got, _ = Q.attn_norm_rope(q, None, positions=pos, inv_freq=f, axes=axes)
    assert Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG
    axes[3] = axes[9] = 0
    assert torch.equal(got, Q.attn_norm_rope(q, None, positions=pos, inv_freq=f, axes=axes)[0])


def test_norm_rope_captured(Q):
    """Captured on a side stream, replayed with other inputs."""
    case = (65, 8, 2, 128, 128, 1, False, BF16, BF16, 1 << 20)
    wide, q, k, qw, kw, pos, f, axes = inputs(Q, case, 4, "slice")
    out = tuple(torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (q, k))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.attn_norm_rope(q, k, qw, kw, pos, f, out=out)
    for _ in range(3):
        wide.normal_()
        pos.add_(1000)
        graph.replay()
        for y, x, w in zip(out, (q, k), (qw, kw)):
            near(y, *norm_rope64(x, w, pos, f, None, 1e-6, False))


def test_norm_rope_refusals(Q):
    q, k = torch.randn((4, 2, 64), device="cuda"), torch.randn((4, 1, 64), device="cuda")
    w, pos, f = torch.ones(64, device="cuda"), torch.arange(4, device="cuda"), Q.rope_inv_freq(64, device="cuda")
    good = dict(q=q, k=k, q_weight=w, k_weight=w, positions=pos, inv_freq=f)
    Q.attn_norm_rope(**good)
    two = torch.stack([pos, pos])
    for kw in (dict(k=k.half()), dict(k=k[:3]), dict(k=k[:, :0]), dict(q=q.cpu()), dict(q_weight=w.half()), dict(q_weight=w[:32]),
               dict(q_weight=w.double()), dict(positions=pos.int()), dict(positions=two), dict(positions=pos[:3]),
               dict(positions=None), dict(inv_freq=f.float()), dict(axes=torch.zeros(31, dtype=torch.int32, device="cuda")),
               dict(positions=two, axes=torch.zeros(32, device="cuda")), dict(k=None), dict(eps=-1.0), dict(mscale=0.0),
               dict(out=(q, torch.empty_like(q))), dict(out=(k, k)), dict(out=(torch.empty_like(q), q[:, :1])),
               dict(q=q[..., ::2]), dict(q_weight=None, k_weight=None, positions=None, inv_freq=None)):
        with pytest.raises((Q.Q8AttnError, ValueError, TypeError)):
            Q.attn_norm_rope(**{**good, **kw})
