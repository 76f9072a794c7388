"""Rotary positions, the paged Q8_0 cache and the attention over it, against plain
64-bit implementations.

Tolerances.  An output is rounded once to its type: u = finfo.eps / 2 of its value.
Rotation: products and sums in fp32, each off by 2^-24, angles by pi 2^-25 and
sincospif's 2^-23, so 2^-22 (|a| + |b|) in all, plus the fp64 table's 2^-51 of the
angle.  Attention: every weight is rounded once to fp16 (2^-11); a score is formed
by at most 16 fp32 operations of 2^-23 each on terms bounded by G = scale sum |q||k|,
and e^x turns a score's absolute error into a weight's relative one, in the numerator
and the denominator; so an output is within
  (2^-11 + 2 (2^-19 G + 2^-21)) A + u |y|,  A = sum p |v| / sum p,
with 2^-11 once more where the values are rounded to fp16 as well (bf16 outputs, whose own
rounding is 2^-8).  A sequence of more than 64 rows per K/V head also counts, in the sum of
its weights l, the largest weight of each key tile as it was rounded: l' = l + sum over tiles
of e_t w_t with |e_t| <= 2^-11 and sum w_t <= l, so |l' - l| <= 2^-11 l and the quotient
moves by at most 2^-11 |y| more; and its weights, between 2^7 and 2^15 at the row's largest
score, are off by half a subnormal step, 2^-25, where they are below fp16's normal range: by
2^-32 sum |v| of the output.
"""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import q8_0

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


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ rotary --


def rope64(x, positions, inv_freq, interleaved, mscale=1.0, inverse=False):
    """The formula in 64 bits (CPU), and the bound of its fp32 evaluation."""
    x = x.double().cpu()
    rot = 2 * len(inv_freq)
    turns = positions.cpu().double()[:, None] * inv_freq.cpu()
    c, s = turns.cos()[:, None] * mscale, turns.sin()[:, None] * mscale * (-1 if inverse else 1)
    first = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    second = first + (1 if interleaved else rot // 2)
    a, b = x[..., first], x[..., second]
    y, bound = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    e = (2.0 ** -22 + 2.0 ** -51 * turns.abs()[:, None]) * (a.abs() + b.abs()) * abs(mscale)
    bound[..., first] = bound[..., second] = e
    return y, bound


ROPE_CASES = [
    # tokens, heads, D, rot, interleaved, dtype, largest position
    (1, 1, 64, 64, False, F16, 10),
    (1, 1, 64, 2, True, F32, 10),
    (7, 5, 128, 128, True, BF16, 1 << 20),
    (33, 3, 128, 96, False, F16, 1 << 31),
    (5, 32, 64, 32, True, F16, 1 << 17),
    (64, 32, 64, 64, False, F32, 1 << 20),
    (9, 2, 64, 24, False, BF16, 5000),      # rot / 2 not a multiple of the 16-byte access
    (9, 2, 128, 10, True, F16, 5000),
    (1030, 3, 128, 64, False, BF16, 1 << 20),
    (2051, 1, 64, 48, True, F32, 1 << 16),
]


@pytest.mark.parametrize("tokens,heads,D,rot,inter,dtype,far", ROPE_CASES)
@pytest.mark.parametrize("form", ["fresh", "slice", "in place", "odd offset"])
def test_rope(Q, tokens, heads, D, rot, inter, dtype, far, form):
    g = gen(1)
    wide = torch.randn((tokens, 3 * heads + 1, D), generator=g, device="cuda").to(dtype)
    if form == "fresh":
        x = wide[:, :heads].contiguous()
    elif form == "odd offset":   # element-aligned only
        flat = torch.empty(tokens * heads * D + 1, dtype=dtype, device="cuda")
        x = flat[1:].view(tokens, heads, D)
        x.copy_(wide[:, :heads])
    else:
        x = wide[:, heads:2 * heads]
    pos = torch.randint(-far, far, (tokens,), generator=g, device="cuda")
    f = Q.rope_inv_freq(rot, factor=1.5, device="cuda")
    want, bound = rope64(x, pos, f, inter, 0.75)
    before = wide.clone()
    out = Q.attn_rope(x, pos, f, interleaved=inter, mscale=0.75, out=x if form == "in place" else None)
    got = out.double().cpu()
    assert ((got - want).abs() <= bound + unit(dtype) * (want.abs() + bound) + 2.0 ** -25).all()
    if form == "in place":
        keep = [h for h in range(3 * heads + 1) if not heads <= h < 2 * heads]
        assert torch.equal(wide[:, keep], before[:, keep])
    else:
        assert torch.equal(wide, before)
    assert torch.equal(out[..., rot:], before[:, :heads][..., rot:] if form in ("fresh", "odd offset")
                       else before[:, heads:2 * heads][..., rot:])


def test_rope_gradient(Q):
    """The inverse is the transpose: it is the gradient of <rope(x), w> in x, by the formula and by
    differences (the rotation is linear, so a difference of 1 is exact up to rounding)."""
    g = gen(2)
    x = torch.randn((3, 2, 64), generator=g, device="cuda")
    w = torch.randn((3, 2, 64), generator=g, device="cuda")
    pos = torch.tensor([0, 77, 100003], device="cuda")
    f = Q.rope_inv_freq(32, device="cuda")
    grad = Q.attn_rope(w, pos, f, inverse=True, mscale=1.25)
    want, bound = rope64(w, pos, f, False, 1.25, inverse=True)
    assert ((grad.double().cpu() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all()
    base = Q.attn_rope(x, pos, f, mscale=1.25).double()
    for t, h, c in [(0, 0, 0), (1, 1, 5), (2, 0, 21), (2, 1, 31), (1, 0, 40)]:
        moved = x.clone()
        moved[t, h, c] += 1.0
        diff = ((Q.attn_rope(moved, pos, f, mscale=1.25).double() - base) * w.double()).sum().item()
        assert abs(diff - grad[t, h, c].item()) <= 64 * 2.0 ** -20


# ------------------------------------------------------------------- pages --


def empty_pages(n_pages, heads, page, D, fill=0xA5):
    return torch.full((n_pages, heads, page, D // 32 * 34), fill, dtype=torch.uint8, device="cuda")


def rows_of(x):
    """Q8_0 rows [T, H, bytes] of fp32-valued x [T, H, D], by the oracle."""
    x = x.float().cpu().numpy()
    return torch.from_numpy(q8_0.quantize_kv(x[None])[0].transpose(1, 0, 2).copy())


def at_slots(pages, slots):
    page = pages.shape[2]
    return pages[slots // page, :, slots % page]


APPEND_CASES = [
    # tokens, heads, D, page, dtype
    (1, 1, 64, 16, F32), (1, 8, 128, 16, F16), (17, 3, 64, 16, BF16), (15, 5, 128, 64, F32),
    (64, 8, 128, 16, BF16), (300, 2, 64, 256, F16), (33, 32, 64, 32, F32),
]


@pytest.mark.parametrize("tokens,heads,D,page,dtype", APPEND_CASES)
@pytest.mark.parametrize("slices", [False, True])
def test_append_bytes(Q, tokens, heads, D, page, dtype, slices):
    """Without rotation every byte is the oracle's; skipped tokens and all other bytes stay."""
    g = gen(3)
    qkv = (torch.randn((tokens, 3 * heads, D), generator=g, device="cuda") * 3).to(dtype)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    if not slices:
        k, v = k.contiguous(), v.contiguous()
    n_pages = tokens // page + 3
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:tokens]
    slots[::5] = -1 - slots[::5]
    kp, vp = empty_pages(n_pages, heads, page, D), empty_pages(n_pages, heads, page, D, 0x3C)
    wk, wv = kp.clone(), vp.clone()
    kept = slots >= 0
    for pages, x in ((wk, k), (wv, v)):
        pages[slots[kept] // page, :, slots[kept] % page] = rows_of(x).cuda()[kept]
    Q.q8kv_append_paged(k, v, kp, vp, slots)
    assert torch.equal(kp, wk) and torch.equal(vp, wv)


@pytest.mark.parametrize("tokens,heads,D,page,dtype", APPEND_CASES)
@pytest.mark.parametrize("rot,inter", [(64, False), (64, True), (32, False), (20, False), (6, True), (48, True)])
def test_append_rotated(Q, tokens, heads, D, page, dtype, rot, inter):
    """Rotated keys: the bytes are those of quantising attn_rope's fp32 result, and the values are
    within half a code of the formula's."""
    g = gen(4)
    k = torch.randn((tokens, heads, D), generator=g, device="cuda").to(dtype)
    v = torch.randn((tokens, heads, D), generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda")
    f = Q.rope_inv_freq(rot, device="cuda")
    n_pages = tokens // page + 2
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:tokens]
    kp, vp = empty_pages(n_pages, heads, page, D), empty_pages(n_pages, heads, page, D)
    Q.q8kv_append_paged(k, v, kp, vp, slots, pos, f, interleaved=inter, mscale=1.5)
    turned = Q.attn_rope(k.float(), pos, f, interleaved=inter, mscale=1.5)
    assert torch.equal(at_slots(kp, slots).cpu(), rows_of(turned))
    assert torch.equal(at_slots(vp, slots).cpu(), rows_of(v))
    want, bound = rope64(k, pos, f, inter, 1.5)
    got = torch.from_numpy(q8_0.dequantize_kv(at_slots(kp, slots).cpu().numpy()))
    scale = torch.from_numpy(q8_0.unpack_rows(at_slots(kp, slots).cpu().numpy(), D // 32)[0].astype(np.float64))
    half = scale.repeat_interleave(32, -1) * (0.5 + 127 * 2.0 ** -11)   # the scale itself is rounded to fp16
    assert ((got - want).abs() <= half + bound + 2.0 ** -22 * want.abs()).all()


@pytest.mark.parametrize("D,heads,page", [(64, 3, 16), (128, 8, 128), (64, 1, 4096)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("tokens", [1, 31, 257])
def test_read(Q, D, heads, page, dtype, tokens):
    """Values in any order, repeats among them; a negative slot leaves its row."""
    g = gen(5)
    kp = torch.randint(0, 256, (4, heads, page, D // 32 * 34), generator=g, device="cuda").to(torch.uint8)
    vp = kp.flip(0).contiguous()
    for p in (kp, vp):   # scales: finite, of any size
        p.unflatten(-1, (-1, 34))[..., 1] &= 0x3B
    slots = torch.randint(0, 4 * page, (tokens,), generator=g, device="cuda")
    slots[-1] = slots[0]
    slots[3::7] = -5
    out = tuple(torch.full((tokens, heads, D), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    Q.q8kv_read_paged(kp, vp, slots, dtype, out=out)
    for pages, got in zip((kp, vp), out):
        want = torch.from_numpy(q8_0.dequantize_kv(at_slots(pages, slots.clamp(min=0)).cpu().numpy())).to(dtype)
        want[slots.cpu() < 0] = 7.0
        assert torch.equal(got.cpu(), want)


# --------------------------------------------------------------- attention --


class Batch:
    """Sequences in pages, with every byte that no key owns set to values that must not matter."""

    def __init__(self, q_lens, kv_lens, heads, kv_heads, D, page, dtype, seed=0, q_scale=1.0, v_scale=1.0, spare=1,
                 stray_rows=0, table_extra=2, interleave_pools=False):
        g = gen(seed)
        self.q_lens, self.kv_lens_host = list(q_lens), list(kv_lens)
        self.group, self.D, self.page = heads // kv_heads, D, page
        self.n_rows = sum(q_lens)
        self.q = (torch.randn((self.n_rows + stray_rows, heads, D), generator=g, device="cuda") * q_scale).to(dtype)
        used = [-(-n // page) for n in kv_lens]
        n_pages = sum(used) + spare
        rb = D // 32 * 34
        if interleave_pools:
            both = torch.empty((n_pages, 2, kv_heads, page, rb), dtype=torch.uint8, device="cuda")
            self.k_pages, self.v_pages = both[:, 0], both[:, 1]
        else:
            self.k_pages = torch.empty((n_pages, kv_heads, page, rb), dtype=torch.uint8, device="cuda")
            self.v_pages = torch.empty_like(self.k_pages)
        for p in (self.k_pages, self.v_pages):   # scales of NaN and infinity where nothing is kept
            junk = torch.randint(0, 256, p.shape, generator=g, device="cuda").to(torch.uint8)
            blocks = junk.unflatten(-1, (-1, 34))
            blocks[..., 0] = torch.where(blocks[..., 2] > 127, 0, 1)
            blocks[..., 1] = 0x7C
            p.copy_(junk)
        order = torch.randperm(n_pages, generator=g, device="cuda").int()
        width = max(used) + table_extra
        self.table = torch.full((len(q_lens), width), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
        self.k, self.v, first = [], [], 0
        for b, n in enumerate(kv_lens):
            self.table[b, :used[b]] = order[first:first + used[b]]
            first += used[b]
            kv = [(torch.randn((n, kv_heads, D), generator=g, device="cuda") * s).cpu() for s in (1.0, v_scale)]
            slots = self.slots(b, torch.arange(n, device="cuda"))
            for pages, x, keep in zip((self.k_pages, self.v_pages), kv, (self.k, self.v)):
                rows = rows_of(x)
                pages[slots // page, :, slots % page] = rows.cuda()
                keep.append(torch.from_numpy(q8_0.dequantize_kv(rows.numpy())))
        self.kv_lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
        self.cu_q = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device="cuda")

    def slots(self, b, at):
        return self.table[b, at // self.page].long() * self.page + at % self.page

    def args(self):
        return (self.q, self.k_pages, self.v_pages, self.table, self.kv_lens, self.cu_q, max(max(self.q_lens), 1),
                max(self.kv_lens_host))

    def check(self, out, causal=True, scale=None, sequences=None):
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        u = unit(out.dtype)
        row = 0
        for b, (nq, n) in enumerate(zip(self.q_lens, self.kv_lens_host)):
            if nq == 0 or (sequences is not None and b not in sequences):
                row += nq
                continue
            q = self.q[row:row + nq].double()
            k, v = self.k[b].cuda(), self.v[b].cuda()
            seen = torch.arange(n, device="cuda")[None] <= (torch.arange(nq, device="cuda")[:, None] + n - nq
                                                           if causal else n)
            for h in range(q.shape[1]):
                kh = h // self.group
                s = q[:, h] @ k[:, kh].T * scale
                G = (q[:, h].abs() @ k[:, kh].abs().T * scale).amax() if n else 0.0
                p = torch.where(seen, s, -math.inf)
                top = p.amax(1, keepdim=True) if n else torch.zeros((nq, 1), device="cuda")
                p = torch.exp(p - torch.where(top == -math.inf, 0, top))
                p = torch.nan_to_num(p, nan=0.0)
                total = p.sum(1, keepdim=True)
                p = p / torch.where(total == 0, 1, total)
                y, A = p @ v[:, kh], p @ v[:, kh].abs()
                got = out[row:row + nq, h].double()
                weights = 2.0 ** -11 * (1 if out.dtype == F16 else 2)
                tol = (weights + 2 * (2.0 ** -19 * G + 2.0 ** -21)) * A
                if nq * self.group > 64:
                    tol = tol + 2.0 ** -11 * y.abs() + 2.0 ** -32 * (seen.double() @ v[:, kh].abs())
                tol = tol + u * (y.abs() + tol) + 2.0 ** -25
                bad = ~((got - y).abs() <= tol)
                assert not bad.any(), (b, h, int(bad.sum()), float((got - y).abs().max()), float(tol.max()))
            row += nq


FEW = [
    # new tokens, keys, heads, kv heads, D, page
    ([1], [1], 1, 1, 64, 16),
    ([1], [1], 4, 4, 128, 16),
    ([1], [31], 8, 8, 64, 16),
    ([1], [32], 8, 1, 64, 16),
    ([1], [33], 4, 2, 64, 32),
    ([1], [255], 8, 2, 128, 16),
    ([1], [2049], 32, 8, 128, 64),
    ([1], [20011], 8, 8, 64, 128),
    ([1, 1, 1, 1, 1], [1, 700, 16, 0, 4097], 8, 2, 64, 16),
    ([1, 0, 1, 1], [300, 50, 17, 1000], 12, 4, 128, 32),
    ([2, 3, 1, 5], [2, 3, 900, 77], 4, 2, 64, 16),
    ([8], [513], 8, 8, 128, 256),
    ([16, 9], [1000, 9], 8, 2, 64, 64),
    ([7, 30], [100, 3001], 16, 2, 128, 16),
    ([64], [640], 4, 4, 64, 32),
    ([5, 4], [3, 2], 2, 1, 64, 16),        # more new tokens than keys: rows that see none
    ([1] * 300, [(37 * i) % 190 for i in range(300)], 4, 4, 64, 16),
    ([3], [100], 9, 3, 64, 16),
    ([11], [500], 3, 1, 128, 64),
]


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,D,page", FEW)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_few_rows(Q, q_lens, kv_lens, heads, kv_heads, D, page, dtype, causal):
    x = Batch(q_lens, kv_lens, heads, kv_heads, D, page, dtype, seed=len(q_lens) + sum(kv_lens))
    x.check(Q.attn_paged(*x.args(), causal=causal), causal)


MANY = [
    ([128], [128], 2, 2, 64, 16),
    ([129], [129], 1, 1, 128, 16),
    ([300], [300], 4, 2, 64, 128),
    ([513], [1500], 4, 1, 128, 64),
    ([1025, 1, 77], [1025, 600, 2000], 4, 4, 64, 32),
    ([200, 333, 0, 65], [1000, 333, 10, 70], 6, 2, 128, 16),
    ([90], [3000], 8, 2, 64, 256),
    ([100, 5], [40, 5], 5, 1, 64, 16),
    ([257], [4001], 3, 1, 64, 128),
    ([700], [700], 7, 1, 128, 32),
]


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,D,page", MANY)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_many_rows(Q, q_lens, kv_lens, heads, kv_heads, D, page, dtype, causal):
    x = Batch(q_lens, kv_lens, heads, kv_heads, D, page, dtype, seed=len(q_lens) + sum(kv_lens))
    x.check(Q.attn_paged(*x.args(), causal=causal), causal)


@pytest.mark.parametrize("q_len", [1, 20, 300])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_range_of_values(Q, q_len, D, dtype):
    """Sharp softmaxes, large and tiny values and queries."""
    for q_scale, v_scale, scale in [(12.0, 1.0, None), (1.0, 3000.0, None), (1.0, 2e-4, None), (2e-3, 1.0, 5.0)]:
        x = Batch([q_len], [777], 4, 2, D, 16, dtype, seed=5, q_scale=q_scale, v_scale=v_scale)
        x.check(Q.attn_paged(*x.args(), scale=scale), scale=scale)


@pytest.mark.parametrize("q_len", [1, 200])
def test_attention_leaves_other_rows_and_pools_interleaved(Q, q_len):
    x = Batch([q_len, 2], [400, 50], 8, 2, 64, 32, F16, stray_rows=5, interleave_pools=True)
    out = torch.full_like(x.q, 9.0)
    wide = torch.empty((x.q.shape[0], 12, 64), dtype=F16, device="cuda")
    wide[:, 2:10] = x.q
    Q.attn_paged(wide[:, 2:10], *x.args()[1:], out=out)
    x.check(out)
    assert (out[x.n_rows:] == 9.0).all()
    assert torch.equal(out, Q.attn_paged(*x.args(), out=torch.full_like(x.q, 9.0)))


@pytest.mark.parametrize("q_len,dtype", [(1, F16), (200, BF16)])
def test_attention_repeats_and_streams(Q, q_len, dtype):
    """The same bits every time, also on another stream and with a caller's workspace of any contents."""
    x = Batch([q_len, q_len], [9000, 1200], 8, 2, 128, 64, dtype)
    first = Q.attn_paged(*x.args())
    n = Q.paged_workspace_floats(2, 2 * q_len, 8, 2, q_len, 9000, 128)
    ws = torch.full((n,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        second = Q.attn_paged(*x.args(), workspace=ws)
        third = Q.attn_paged(*x.args(), workspace=ws)
    s.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third)


def test_attention_nan_and_infinite_queries_stay_in_their_rows(Q):
    for q_len in (4, 200):
        x = Batch([q_len, 3], [300, 300], 4, 2, 64, 16, F16)
        want = Q.attn_paged(*x.args())
        x.q[1, 0, 5] = float("nan")
        x.q[2, 3, 5] = float("inf")
        got = Q.attn_paged(*x.args())
        touched = torch.zeros_like(got, dtype=torch.bool)
        touched[1, 0] = touched[2, 3] = True
        assert torch.isnan(got[1, 0]).all()
        assert torch.equal(got[~touched], want[~touched])


@pytest.mark.parametrize("q_len", [1, 200])
def test_bad_indices_are_recorded(Q, q_len):
    """Out-of-range pages, lengths and offsets are never followed; the other sequences' results hold."""
    x = Batch([q_len, q_len], [500, 300], 4, 2, 64, 16, F16)
    cases = []
    for bad in (x.k_pages.shape[0], -1, 0x7FFFFFFF):
        table = x.table.clone()
        table[0, 3] = bad
        cases.append((table, x.kv_lens, x.cu_q, True))
    lens = x.kv_lens.clone()
    lens[0] = x.table.shape[1] * x.page + 1
    table = x.table.clamp(max=x.k_pages.shape[0] - 1)
    cases.append((table, lens, x.cu_q, True))
    lens = x.kv_lens.clone()
    lens[0] = -4
    cases.append((x.table, lens, x.cu_q, True))
    cu = x.cu_q.clone()
    cu[2] += 1
    cases.append((x.table, x.kv_lens, cu, False))
    for table, lens, cu, other in cases:
        got = Q.attn_paged(x.q, x.k_pages, x.v_pages, table, lens, cu, q_len, 500)
        torch.cuda.synchronize()
        assert Q.status() == Q.Q8A_ERR_INVALID_ARG
        rc, word = Q.device_status(clear=True)
        assert rc == Q.Q8A_ERR_INVALID_ARG and word & 2
        assert Q.status() == 0
        if other:
            # how a sequence's keys are shared out depends on the others' lengths, so its last bits may too
            x.check(got, sequences=[1])
    slots = torch.tensor([0, 16 * x.k_pages.shape[0], 1 << 50], device="cuda")
    k = torch.randn((3, 2, 64), device="cuda")
    kp, vp = x.k_pages.clone(), x.v_pages.clone()
    Q.q8kv_append_paged(k, k, kp, vp, slots)
    assert Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG
    out = Q.q8kv_read_paged(kp, vp, slots, F32)
    assert Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG
    assert torch.equal(kp[0, :, 1:], x.k_pages[0, :, 1:]) and torch.equal(kp[1:], x.k_pages[1:])
    assert torch.equal(kp[0, :, 0].cpu(), rows_of(k[:1])[0]) and len(out) == 2


# ------------------------------------------------------------ used together --


def serve(Q, D, heads, kv_heads, page, dtype, prompts, steps, inter, plan):
    """Prompts in chunks, then single tokens, as a server runs them: rotate, append, attend."""
    g = gen(9)
    B, n = len(prompts), [p + steps for p in prompts]
    rot = D // 2
    f = Q.rope_inv_freq(rot, factor=2.0, device="cuda")
    width = max(-(-m // page) for m in n)
    table = torch.randperm(B * width, generator=g, device="cuda").int().view(B, width)
    kp, vp = (empty_pages(B * width, kv_heads, page, D, 0xFF) for _ in range(2))
    qkv = [torch.randn((m, heads + 2 * kv_heads, D), generator=g, device="cuda").to(dtype) for m in n]
    done, outs = [0] * B, [[] for _ in range(B)]
    for counts in plan:
        take = [(b, c) for b, c in enumerate(counts) if c]
        x = torch.cat([qkv[b][done[b]:done[b] + c] for b, c in take])
        pos = torch.cat([torch.arange(done[b], done[b] + c, device="cuda") for b, c in take])
        seq = torch.cat([torch.full((c,), b, device="cuda") for b, c in take])
        slots = table[seq, pos // page].long() * page + pos % page
        q = Q.attn_rope(x[:, :heads], pos, f, interleaved=inter)
        Q.q8kv_append_paged(x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], kp, vp, slots, pos, f,
                            interleaved=inter)
        for b, c in take:
            done[b] += c
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        y = Q.attn_paged(q, kp, vp, table, lens, cu, max(counts), max(done))
        row = 0
        for b, c in take:
            outs[b].append(y[row:row + c])
            row += c
    return qkv, f, kp, vp, table, [torch.cat(o) for o in outs]


@pytest.mark.parametrize("D,heads,kv_heads,page,dtype,inter",
                         [(64, 8, 8, 16, F16, False), (128, 8, 2, 64, BF16, True), (64, 6, 2, 32, BF16, False)])
def test_a_served_batch(Q, D, heads, kv_heads, page, dtype, inter):
    prompts, steps = [150, 37, 300], 4
    plan = [[100, 37, 200], [50, 0, 100]] + [[1, 1, 1]] * steps
    qkv, f, kp, vp, table, outs = serve(Q, D, heads, kv_heads, page, dtype, prompts, steps, inter, plan)
    x = Batch.__new__(Batch)
    x.group, x.D, x.page, x.table = heads // kv_heads, D, page, table
    x.q_lens = x.kv_lens_host = [p + steps for p in prompts]
    x.q = torch.cat([Q.attn_rope(t[:, :heads], torch.arange(len(t), device="cuda"), f, interleaved=inter) for t in qkv])
    x.k, x.v = [], []
    for b, n in enumerate(x.kv_lens_host):   # the cache's values, which the append's own tests hold to the formula
        slots = x.slots(b, torch.arange(n, device="cuda"))
        for pages, keep in ((kp, x.k), (vp, x.v)):
            keep.append(torch.from_numpy(q8_0.dequantize_kv(at_slots(pages, slots).cpu().numpy())))
        k32, v32 = Q.q8kv_read_paged(kp, vp, slots, F32)
        assert torch.equal(k32.cpu().double(), x.k[b]) and torch.equal(v32.cpu().double(), x.v[b])
        turned, _ = rope64(qkv[b][:, heads:heads + kv_heads], torch.arange(n), f.cpu(), inter)
        assert (x.k[b] - turned).abs().max() < 0.03   # amax / 254 of values below 7
    x.check(torch.cat(outs))


def test_pages_of_the_planes(Q):
    """A plane of q8kv_quantize is a sequence of pages: the chunk steps and the paged attention agree."""
    g = gen(11)
    M, H, D, page = 640, 4, 64, 128
    k, v = (torch.randn((1, M, H, D), generator=g, device="cuda") for _ in range(2))
    q = torch.randn((1, M, H, D), generator=g, device="cuda").half()
    out, k8, v8 = Q.prefill_attention(q, k, v, 256)
    pages = [p[0, :, :M * 68].view(H, M // page, page, 68).transpose(0, 1).contiguous() for p in (k8, v8)]
    table = torch.arange(M // page, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([M], dtype=torch.int32, device="cuda")
    got = Q.attn_paged(q[0], *pages, table, lens, torch.tensor([0, M], dtype=torch.int32, device="cuda"), M, M)
    # each side is within its weights' rounding (2^-11 of at most |v| < 6) and the output's
    assert (got.float() - out[0].float()).abs().max() <= 2 * (2.0 ** -11 + 2.0 ** -13) * 6
    assert (got.float() - out[0].float()).norm() <= 1e-3 * out.float().norm()


def test_captured_step_replays_with_new_lengths(Q):
    """One captured step (rotate, append, attend) replayed as sequences grow; a padded row is skipped."""
    g = gen(12)
    B, H, HK, D, page, width = 4, 8, 2, 64, 16, 40
    dtype, f = BF16, Q.rope_inv_freq(64, device="cuda")
    kp, vp = (empty_pages(B * width, HK, page, D, 0xFF) for _ in range(2))
    table = torch.randperm(B * width, generator=g, device="cuda").int().view(B, width)
    kept = torch.randn((2, B * width * page, HK, D), generator=g, device="cuda")   # the sequences' earlier rows
    Q.q8kv_append_paged(kept[0], kept[1], kp, vp, torch.arange(B * width * page, device="cuda"))
    x = torch.randn((B, H + 2 * HK, D), generator=g, device="cuda").to(dtype)
    pos = torch.zeros(B, dtype=torch.int64, device="cuda")
    slots = torch.full((B,), -1, dtype=torch.int64, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    out = torch.zeros((B, H, D), dtype=dtype, device="cuda")
    ws = torch.empty(Q.paged_workspace_floats(B, B, H, HK, 1, width * page, D), device="cuda")
    qr = torch.empty((B, H, D), dtype=dtype, device="cuda")

    def step():
        Q.attn_rope(x[:, :H], pos, f, out=qr)
        Q.q8kv_append_paged(x[:, H:H + HK], x[:, H + HK:], kp, vp, slots, pos, f)
        Q.attn_paged(qr, kp, vp, table, lens, cu, 1, width * page, out=out, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    mirror = [kp.clone(), vp.clone()]
    for i in range(30):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(dtype))
        n = torch.tensor([i, 2 * i, 20 * i if i < 30 else 0, 0], device="cuda")   # keys before this step
        pos.copy_(n)
        at = table[torch.arange(B, device="cuda"), n // page].long() * page + n % page
        at[3] = -1                                                                # padding
        slots.copy_(at)
        lens.copy_(torch.where(at >= 0, n + 1, 0))
        graph.replay()
        got = out.clone()
        q = Q.attn_rope(x[:, :H], pos, f)
        Q.q8kv_append_paged(x[:, H:H + HK], x[:, H + HK:], *mirror, slots, pos, f)
        assert torch.equal(kp, mirror[0]) and torch.equal(vp, mirror[1])
        assert torch.equal(got, Q.attn_paged(q, kp, vp, table, lens, cu, 1, width * page))
        assert (got[3] == 0).all()


@pytest.mark.parametrize("q_lens,kv_lens", [([300, 1, 60], [300, 700, 900]), ([100, 20], [5000, 300]), ([9], [70])])
def test_captured_prompts_replay(Q, q_lens, kv_lens):
    """A captured call over prompts, replayed after the lengths shrink; two graphs of one stream share a workspace."""
    x = Batch(q_lens, kv_lens, 8, 2, 64, 32, F16, seed=21)
    y = Batch(q_lens[::-1], kv_lens[::-1], 8, 2, 64, 32, F16, seed=22)
    n = Q.paged_workspace_floats(len(q_lens), x.n_rows, 8, 2, max(q_lens), max(kv_lens), 64)
    ws = torch.empty(max(n, 1), device="cuda")
    outs, graphs = [torch.zeros_like(b.q) for b in (x, y)], []
    for b, out in zip((x, y), outs):
        Q.attn_paged(*b.args(), out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            Q.attn_paged(*b.args(), out=out, workspace=ws)
        graphs.append(graph)
    for _ in range(3):
        for out in outs:
            out.fill_(5.0)
        graphs[0].replay()
        graphs[1].replay()
        x.check(outs[0])
        y.check(outs[1])
    # shorter sequences within the captured bounds: the first keeps its first rows' keys only
    drop = q_lens[0] // 2
    x.kv_lens[0] -= drop
    x.cu_q[1:] -= drop
    outs[0].fill_(5.0)
    graphs[0].replay()
    short = Q.attn_paged(x.q, x.k_pages, x.v_pages, x.table, x.kv_lens, x.cu_q, max(q_lens), max(kv_lens),
                         out=torch.full_like(x.q, 5.0))
    assert torch.equal(outs[0], short)
    assert (outs[0][x.n_rows - drop:] == 5.0).all()


@pytest.mark.parametrize("tokens", [1, 40, 700])
def test_calls_in_a_row_see_each_others_writes(Q, tokens):
    """The same rows are written, read back, attended to and written again without a wait of the host between:
    each call sees what the call before it wrote."""
    H, D, page, steps = 4, 64, 16, 60
    n_pages = -(-tokens // page)
    shape = (n_pages, H, page, 68)
    kp, vp = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(tokens, device="cuda")
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    q = torch.ones((1, H, D), dtype=F16, device="cuda")
    vals = [torch.full((tokens, H, D), 127.0 * 2 ** -6 * (i + 1), dtype=F32, device="cuda") for i in range(steps)]
    outs = [tuple(torch.empty((tokens, H, D), dtype=F32, device="cuda") for _ in range(2)) for _ in range(steps)]
    att = [torch.empty_like(q) for _ in range(steps)]
    ws = torch.empty(max(Q.paged_workspace_floats(1, 1, H, H, 1, tokens, D), 4), device="cuda")
    torch.cuda.synchronize()
    for i in range(steps):
        Q.q8kv_append_paged(vals[i], vals[i], kp, vp, slots)
        Q.q8kv_read_paged(kp, vp, slots, F32, out=outs[i])
        Q.attn_paged(q, kp, vp, table, lens, cu, 1, tokens, out=att[i], workspace=ws)
    torch.cuda.synchronize()
    for i in range(steps):
        # amax / 127 = 2^-6 (i + 1) exactly, so every code is 127 and every value exact; equal values average to
        # themselves but for the weights' rounding (2^-11 each way) and the output's
        assert torch.equal(outs[i][0], vals[i]) and torch.equal(outs[i][1], vals[i]), i
        x = float(vals[i][0, 0, 0])
        assert (att[i].double() - x).abs().max() <= 3 * 2.0 ** -11 * x, i


def test_two_streams_at_once(Q):
    """Independent calls on two streams, each with its own workspace."""
    a = Batch([1, 1], [40000, 3000], 8, 2, 128, 64, BF16, seed=31)
    b = Batch([400], [2000], 4, 2, 64, 16, F16, seed=32)
    want = [Q.attn_paged(*x.args()) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s, x in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(Q.attn_paged(*x.args()))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])
    a.check(want[0])
    b.check(want[1])


def guarded(shape, dtype, fill=0x5A):
    """A tensor with 256 guard bytes on both sides."""
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    raw = torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda")
    return raw[256:256 + n].view(dtype).view(shape), raw, fill


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [300, 2100]), ([5, 3], [40, 3000]), ([40, 17], [700, 90]),
                                            ([200, 30], [500, 1000]), ([300], [300])])
def test_nothing_is_written_beside_the_buffers(Q, q_lens, kv_lens, D, page):
    x = Batch(q_lens, kv_lens, 8, 2, D, page, F16, seed=41)
    args = x.args()
    pools = (x.k_pages.clone(), x.v_pages.clone())
    out, out_raw, _ = guarded(x.q.shape, F16)
    n = Q.paged_workspace_floats(len(q_lens), x.n_rows, 8, 2, max(q_lens), max(kv_lens), D)
    ws, ws_raw, _ = guarded((max(n, 4),), F32)
    Q.attn_paged(*args, out=out, workspace=ws)
    x.check(out)
    for raw in (out_raw, ws_raw):
        assert (raw[:256] == 0x5A).all() and (raw[-256:] == 0x5A).all()
    assert torch.equal(x.k_pages, pools[0]) and torch.equal(x.v_pages, pools[1])
    # append and rope into guarded buffers
    T = 37
    k = torch.randn((T, 2, D), device="cuda", generator=gen(2))
    pages, raw_k, _ = guarded((3, 2, page, D // 32 * 34), torch.uint8)
    pages_v, raw_v, _ = guarded((3, 2, page, D // 32 * 34), torch.uint8)
    slots = torch.arange(3 * page - T, 3 * page, device="cuda")
    Q.q8kv_append_paged(k, k, pages, pages_v, slots)
    rot, rot_raw, _ = guarded((T, 2, D), F32)
    Q.attn_rope(k, torch.arange(T, device="cuda"), Q.rope_inv_freq(D, device="cuda"), out=rot)
    rd, rd_raw, _ = guarded((T, 2, D), BF16)
    rd2, rd2_raw, _ = guarded((T, 2, D), BF16)
    Q.q8kv_read_paged(pages, pages_v, slots, BF16, out=(rd, rd2))
    for raw in (raw_k, raw_v, rot_raw, rd_raw, rd2_raw):
        assert (raw[:256] == 0x5A).all() and (raw[-256:] == 0x5A).all()
    used = torch.zeros((3, page), dtype=torch.bool, device="cuda")
    used.view(-1)[slots] = True
    assert (pages.transpose(1, 2)[~used] == 0x5A).all() and (pages_v.transpose(1, 2)[~used] == 0x5A).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [700]), ([1], [40000]), ([13], [3000]), ([40, 17], [700, 9000]),
                                            ([300], [4000]), ([600, 700], [600, 700])])
def test_rows_aligned_to_16_bytes_only(Q, q_lens, kv_lens, dtype, D):
    """q, out and the workspace 16 bytes past 32-byte alignment, q's rows an odd number of 16 bytes
    apart: the same bits."""
    x = Batch(q_lens, kv_lens, 4, 2, D, 32, dtype, seed=51)
    want = Q.attn_paged(*x.args())
    x.check(want)
    T, H = x.q.shape[:2]
    stride = H * D + 8
    raw = torch.empty(T * stride + 8, dtype=dtype, device="cuda")
    q = raw[8:].as_strided((T, H, D), (stride, D, 1))
    q.copy_(x.q)
    out = torch.full((T * H * D + 8,), float("nan"), dtype=dtype, device="cuda")[8:].view(T, H, D)
    n = Q.paged_workspace_floats(len(q_lens), T, H, 2, max(q_lens), max(kv_lens), D)
    ws = torch.full((n + 4,), float("nan"), device="cuda")[4:]
    assert all(t.data_ptr() % 32 == 16 for t in ([q, out, ws] if n else [q, out]))
    Q.attn_paged(q, *x.args()[1:], out=out, workspace=ws if n else None)
    assert torch.equal(out, want)


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(Q, seed):
    rng = np.random.default_rng(seed)
    D, page = int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128, 256, 1024]))
    kv_heads = int(rng.integers(1, 4))
    group = int(rng.choice([1, 2, 3, 4, 5, 8]))
    B = int(rng.integers(1, 7))
    top = int(rng.choice([1, 4, 30, 130, 500]))
    q_lens = [int(rng.integers(0, top + 1)) for _ in range(B)]
    if sum(q_lens) == 0:
        q_lens[0] = 1
    kv_lens = [int(n + rng.integers(0, int(rng.choice([2, 100, 4000])))) for n in q_lens]
    if seed % 5 == 0:
        kv_lens[0] = max(0, q_lens[0] - 1)
    kv_lens[-1] = max(kv_lens[-1], 1)
    causal, dtype = bool(rng.random() < 0.7), [F16, BF16][seed % 2]
    x = Batch(q_lens, kv_lens, kv_heads * group, kv_heads, D, page, dtype, seed=seed, interleave_pools=seed % 3 == 0)
    x.check(Q.attn_paged(*x.args(), causal=causal), causal)


def test_offsets_beyond_32_bits(Q):
    """Pages and rows whose byte offsets pass 2^32 (the pools are 5.7 GB each)."""
    D, HK, page, n_pages = 128, 8, 256, 20500
    kp = torch.zeros((n_pages, HK, page, 136), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    g = gen(51)
    at = torch.tensor([n_pages - 1, 3, n_pages - 2], dtype=torch.int32, device="cuda")
    n = 700
    k, v = (torch.randn((n, HK, D), generator=g, device="cuda").half() for _ in range(2))
    pos = torch.arange(n, device="cuda")
    slots = at[pos // page].long() * page + pos % page
    Q.q8kv_append_paged(k, v, kp, vp, slots)
    assert torch.equal(at_slots(kp, slots).cpu(), rows_of(k)) and torch.equal(at_slots(vp, slots).cpu(), rows_of(v))
    k2, v2 = Q.q8kv_read_paged(kp, vp, slots, F32)
    for q_len in (1, 30, 300):
        x = Batch.__new__(Batch)
        x.group, x.D, x.page, x.q_lens, x.kv_lens_host = 2, D, page, [q_len], [n]
        x.q = torch.randn((q_len, 2 * HK, D), generator=g, device="cuda").half()
        x.k, x.v = [k2.double()], [v2.double()]
        out = Q.attn_paged(x.q, kp, vp, at[None], torch.tensor([n], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, q_len], dtype=torch.int32, device="cuda"), q_len, n)
        x.check(out)
    assert kp[:3].count_nonzero() == 0 and vp[4:n_pages - 2].count_nonzero() == 0


def test_binding_refusals(Q):
    """What shapes, types, strides and devices tell is refused before the call."""
    x = Batch([2], [40], 4, 2, 64, 16, F16)
    q, kp, vp, table, lens, cu, mq, mkv = x.args()
    bad = [
        dict(q=q.float()), dict(q=q[:, :, :32]), dict(q=q.transpose(0, 1)), dict(q=q.cpu()), dict(kp=kp.int()),
        dict(kp=kp[:, :, ::2]), dict(kp=kp[:1]), dict(vp=vp[:, :1]), dict(table=table.long()), dict(table=table[0]),
        dict(table=table.t()), dict(lens=lens.long()), dict(lens=lens[:0]), dict(cu=cu[:1]), dict(cu=cu.float()),
        dict(mkv=10 ** 9), dict(mq=-1), dict(scale=0.0), dict(out=q), dict(out=torch.empty_like(q)[:1]),
        dict(out=torch.empty_like(q).float()), dict(workspace=torch.empty(4, device="cuda").half()),
    ]
    for kw in bad:
        a = dict(q=q, kp=kp, vp=vp, table=table, lens=lens, cu=cu, mq=mq, mkv=mkv, scale=None, out=None, workspace=None)
        a.update(kw)
        with pytest.raises(Q.Q8AttnError):
            Q.attn_paged(a["q"], a["kp"], a["vp"], a["table"], a["lens"], a["cu"], a["mq"], a["mkv"], scale=a["scale"],
                         out=a["out"], workspace=a["workspace"])
    f, pos, slots = Q.rope_inv_freq(64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"), \
        torch.zeros(2, dtype=torch.int64, device="cuda")
    for args in [(q.int(), pos, f), (q, pos.int(), f), (q, pos[:1], f), (q, pos, f.float()), (q, pos, f[:0]),
                 (q, pos, torch.cat([f, f])), (q, pos.cpu(), f), (q[..., :32], pos, f)]:
        with pytest.raises(Q.Q8AttnError):
            Q.attn_rope(*args)
    with pytest.raises(Q.Q8AttnError):
        Q.attn_rope(q, pos, f, out=q[:1])
    k = q[:, :2].contiguous()
    for args in [(k, k.float(), kp, vp, slots), (k, k[:1], kp, vp, slots), (q, q, kp, vp, slots),
                 (k, k, kp, vp, slots.int()), (k, k, kp, vp, slots[:1]), (k, k, kp, vp, slots, pos),
                 (k, k, kp, vp, slots, None, f), (k.double(), k.double(), kp, vp, slots)]:
        with pytest.raises(Q.Q8AttnError):
            Q.q8kv_append_paged(*args)
    for args in [(kp, vp, slots.int()), (kp, vp, slots.cpu()), (kp, vp, slots, torch.float64),
                 (kp, vp, slots, F16, (k[:1], k)), (kp, vp[:1], slots)]:
        with pytest.raises(Q.Q8AttnError):
            Q.q8kv_read_paged(*args)
    for kw in (dict(factor=2.0, scaling="base"), dict(factor=2.0, scaling="bands", original_len=100)):
        assert Q.rope_inv_freq(32, device="cuda", **kw).is_cuda
    # empty calls
    assert Q.attn_rope(q[:0], pos[:0], f).shape == (0, 4, 64)
    Q.q8kv_append_paged(k[:0], k[:0], kp, vp, slots[:0])
    assert Q.q8kv_read_paged(kp, vp, slots[:0])[0].shape == (0, 2, 64)
    assert Q.attn_paged(q[:0], kp, vp, table, lens, cu * 0, 0, mkv).shape == (0, 4, 64)
