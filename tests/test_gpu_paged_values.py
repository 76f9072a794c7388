"""attn_paged where values differ by more than a factor of 2^20 between blocks of channels, between keys, and between
what a row sees and what it does not.

Tolerances.  As in Batch.check, with what belongs to the kernel that takes the call.  At most 16 rows per K/V head: a
weight times its block's scale is rounded once to fp16, 2^-11 of it, and V is not rounded.  These products carry
a power of two that puts the largest scale d of the block at 2^6 or more, the largest weight being 1 or more, so below
fp16's normal range they are off by half a step, 2^-25, which is 2^-31 d, times codes of at most 127: together
2^-31 n 127 d of the output, n the keys that the row sees and d their largest scale.  More rows: the products'
terms of Batch.check.  A bound in A covers each score's error too.  Outputs of fp16 are off by half their smallest
step, 2^-25, at least."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import q8_0
from tests import test_gpu_paged as paged
from tests.test_gpu_paged import BF16, F16, Batch, Q, clean_status, rows_of, unit   # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def rewrite(x, b, pages, rows, at):
    """Rows [n, kv_heads, bytes] of keys `at` of sequence b put into its pages."""
    slots = x.slots(b, at.cuda())
    pages[slots // x.page, :, slots % x.page] = rows.cuda()


def set_values(x, b, v):
    """Sequence b's values (fp32 [n, kv_heads, D]) put into its pages."""
    rows = rows_of(v)
    rewrite(x, b, x.v_pages, rows, torch.arange(len(v)))
    x.v[b] = torch.from_numpy(q8_0.dequantize_kv(rows.numpy()))


def check_rows(x, out, causal=True, rows=None, scale=None):
    """Every row (of `rows`, a set of (sequence, token), where given) against the 64-bit result over the keys that it
    sees alone, by a bound per block of channels."""
    most, B = max(x.q_lens), len(x.q_lens)
    # calls of 17 to 128 rows are the tile kernel's, longer ones too but for short sequences that their bounds allow
    short = most * x.group > 128 and (x.q.shape[0] - (B - 1) * most) * x.group <= 16
    u, scale, first = unit(out.dtype), 1 / math.sqrt(x.D) if scale is None else scale, 0
    for b, (nq, n) in enumerate(zip(x.q_lens, x.kv_lens_host)):
        if nq == 0:
            continue
        few = most * x.group <= 16 or (short and nq * x.group <= 16)
        last = torch.arange(nq, device="cuda") + n - nq if causal else torch.full((nq,), n - 1, device="cuda")
        got = out[first:first + nq].double().view(nq, -1, x.group, x.D).permute(1, 2, 0, 3)   # [kv_heads, group, nq, D]
        q = x.q[first:first + nq].double().view(nq, -1, x.group, x.D).permute(1, 2, 0, 3)
        first += nq
        if n == 0:
            assert (got == 0).all()
            continue
        k, v = (t.cuda().transpose(0, 1)[:, None] for t in (x.k[b], x.v[b]))                  # [kv_heads, 1, n, D]
        seen = torch.arange(n, device="cuda") <= last[:, None]
        none, at = last < 0, last.clamp(min=0)
        s = (q @ k.transpose(2, 3) * scale).masked_fill(~seen, -math.inf)
        p = torch.where(none[:, None], 0.0, torch.softmax(s, -1))
        G = torch.where(seen, q.abs() @ k.abs().transpose(2, 3) * scale, 0.0).amax(-1, keepdim=True)
        y, A = p @ v, p @ v.abs()
        score = 2 * (2.0 ** -19 * G + 2.0 ** -21) * A
        if few:
            d = v.abs().unflatten(-1, (-1, 32)).amax(-1).cummax(2).values[:, :, at].repeat_interleave(32, -1)   # 127 d
            tol = 2.0 ** -11 * A + score + 2.0 ** -31 * (last[:, None] + 1) * d
        else:
            tol = (2.0 ** -11 * (1 if out.dtype == F16 else 2) * A + score + 2.0 ** -11 * y.abs() +
                   2.0 ** -32 * v.abs().cumsum(2)[:, :, at])
        tol = torch.where(none[:, None], 0.0, tol + u * (y.abs() + tol) + 2.0 ** -25)
        bad = ~((got - y).abs() <= tol)
        for i in range(nq):
            if rows is not None and (b, i) not in rows:
                bad[:, :, i] = False
        assert not bad.any(), (b, bad.nonzero()[:4].tolist(), float((got - y).abs()[bad].max()),
                               float(((got - y).abs() / tol)[bad].max()))


def sharp(q_lens, kv_lens, heads, kv_heads, D, page, dtype, seed):
    """Few keys carry a row's weight, so that outputs are as large as single values."""
    return Batch(q_lens, kv_lens, heads, kv_heads, D, page, dtype, seed=seed, q_scale=6.0)


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,D,page", paged.FEW + paged.MANY)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("causal", [True, False])
def test_the_bounds_of_the_kernel_that_takes_a_call(Q, q_lens, kv_lens, heads, kv_heads, D, page, dtype, causal):
    """The tile kernel takes calls from 17 rows per K/V head on; up to 16 rows V is not rounded, bf16 or not."""
    x = Batch(q_lens, kv_lens, heads, kv_heads, D, page, dtype, seed=len(q_lens) + sum(kv_lens))
    check_rows(x, Q.attn_paged(*x.args(), causal=causal), causal)


FEW = [([1], [700], 4, 4), ([1, 1], [40, 3000], 8, 2), ([4], [900], 8, 2), ([9], [300], 2, 2), ([16], [16], 1, 1),
       ([1], [9000], 12, 1)]


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads", FEW)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_blocks_of_very_different_scales(Q, q_lens, kv_lens, heads, kv_heads, D, dtype):
    """One block of channels does not cost the others their bits."""
    x = sharp(q_lens, kv_lens, heads, kv_heads, D, 16, dtype, seed=71)
    g = torch.Generator().manual_seed(72)
    lift = torch.tensor([2.0 ** e for e in (12, -13, 0, -6)][:D // 32]).repeat_interleave(32)
    for b, n in enumerate(kv_lens):
        set_values(x, b, torch.randn((n, kv_heads, D), generator=g) * lift)
    check_rows(x, Q.attn_paged(*x.args()))


BURSTS = [
    # new tokens, keys, heads, kv heads: the tokens of a burst in one tile, over two, alone; 2 to 16 rows
    ([4], [900], 8, 2), ([16], [1000], 1, 1), ([16], [33], 1, 1), ([5], [35], 2, 2), ([9], [9], 1, 1), ([4, 3], [64, 2050], 4, 1),
    ([2], [20000], 8, 1), ([8], [4099], 2, 1), ([12, 1, 7], [500, 31, 129], 3, 3), ([7], [4], 2, 1),
]


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads", BURSTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_later_tokens_scale(Q, q_lens, kv_lens, heads, kv_heads, D, dtype):
    """Values that grow by 2^6 or more from token to token of a burst do not touch the rows before them."""
    x = sharp(q_lens, kv_lens, heads, kv_heads, D, 16, dtype, seed=73)
    g = torch.Generator().manual_seed(74)
    for b, (nq, n) in enumerate(zip(q_lens, kv_lens)):
        v = torch.randn((n, kv_heads, D), generator=g) * 2.0 ** -12
        steps = min(nq, n) - 1
        for j in range(steps):   # the keys after the first row's last one
            v[n - steps + j] *= 2.0 ** min(25, 6 * (j + 1) + (j & 1) * 7)
        set_values(x, b, v)
    check_rows(x, Q.attn_paged(*x.args()))


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads", BURSTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("scale,code", [(0x7C00, 0), (0x7C00, 5), (0x7E01, -3)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_infinite_and_nan_scales_that_a_row_does_not_see(Q, q_lens, kv_lens, heads, kv_heads, D, dtype, scale, code, which):
    """A key of a burst with a scale that is no number spoils the rows that see it and no others."""
    x = sharp(q_lens, kv_lens, heads, kv_heads, D, 16, dtype, seed=75)
    pages, blk, clean, first = {"k": x.k_pages, "v": x.v_pages}[which], D // 32 - 1, set(), 0
    spoiled = []
    for b, (nq, n) in enumerate(zip(q_lens, kv_lens)):
        at = max(0, n - max(1, min(nq, n) // 2))   # rows from here on see it
        rows = pages[x.slots(b, torch.tensor([at], device="cuda")) // x.page, :,
                     x.slots(b, torch.tensor([at], device="cuda")) % x.page].cpu().numpy().copy()
        one = rows.reshape(-1, D // 32, 34)
        one[:, blk, :2] = np.frombuffer(np.uint16(scale).tobytes(), dtype=np.uint8)
        one[:, blk, 2:] = np.uint8(code & 0xFF)
        rewrite(x, b, pages, torch.from_numpy(rows), torch.tensor([at]))
        for i in range(nq):
            if n - nq + i >= at:
                spoiled.append(first + i)
            else:
                clean.add((b, i))
        first += nq
    out = Q.attn_paged(*x.args())
    check_rows(x, out, rows=clean)
    if which == "v":
        assert not torch.isfinite(out[spoiled][..., 32 * blk:]).any()
    elif code <= 0:   # an infinite scale times codes whose product with q is below 0 is a score of -inf: weight 0
        assert not torch.isfinite(out[spoiled]).any()


MANY = [
    # 17 rows per K/V head and more: pairs with and without shares, whole CTAs with and without
    ([17], [900], 1, 1), ([40, 17], [700, 90], 2, 2), ([30, 5], [3000, 100], 8, 2), ([32], [20], 4, 1), ([200], [500], 4, 2),
    ([300], [300], 2, 2), ([129, 1, 40], [1000, 200, 40], 3, 3), ([260], [5000], 2, 1), ([70] * 9, [97 * i + 75 for i in range(9)], 20, 20),
]


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads", MANY)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_later_tokens_scale_among_many_rows(Q, q_lens, kv_lens, heads, kv_heads, D, dtype):
    x = sharp(q_lens, kv_lens, heads, kv_heads, D, 16, dtype, seed=77)
    g = torch.Generator().manual_seed(78)
    for b, (nq, n) in enumerate(zip(q_lens, kv_lens)):
        v = torch.randn((n, kv_heads, D), generator=g) * 2.0 ** -12
        v[n - min(nq, n) // 2:] *= 2.0 ** 25
        set_values(x, b, v)
    check_rows(x, Q.attn_paged(*x.args()))


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads", MANY)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("which,scale,code", [("k", 0x7C00, 0), ("k", 0xFE01, -3), ("v", 0x7C00, 0), ("v", 0x7C00, 5),
                                              ("v", 0x7E01, -3), ("v", 0x6400, 127), ("v", 0x6400, 60), ("v", 0x7BFF, 1)])
def test_scales_among_many_rows(Q, q_lens, kv_lens, heads, kv_heads, D, dtype, which, scale, code):
    """Infinite and NaN scales, and scales of V above 515.5, do not touch the rows that do not see them; K's spoil those
    that do."""
    x = sharp(q_lens, kv_lens, heads, kv_heads, D, 16, dtype, seed=79)
    pages, blk, good, first, spoiled = {"k": x.k_pages, "v": x.v_pages}[which], D // 32 - 1, set(), 0, []
    for b, (nq, n) in enumerate(zip(q_lens, kv_lens)):
        at = max(0, n - max(1, min(nq, n) // 2))
        slot = x.slots(b, torch.tensor([at], device="cuda"))
        rows = pages[slot // x.page, :, slot % x.page].cpu().numpy().copy()
        one = rows.reshape(-1, D // 32, 34)
        one[:, blk, :2] = np.frombuffer(np.uint16(scale).tobytes(), dtype=np.uint8)
        one[:, blk, 2:] = np.uint8(code & 0xFF)
        rewrite(x, b, pages, torch.from_numpy(rows), torch.tensor([at]))
        for i in range(nq):
            if n - nq + i < at:
                good.add((b, i))
            else:
                spoiled.append(first + i)
        first += nq
    out = Q.attn_paged(*x.args())
    check_rows(x, out, rows=good)
    if which == "k":
        assert torch.isnan(out[spoiled]).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len", [20, 200])
def test_the_largest_values(Q, q_len, D, dtype):
    """Scales of 515.5, the largest that count: values up to 65,468.5, of both signs, averaged over many keys."""
    x = Batch([q_len], [400], 2, 2, D, 16, dtype, seed=81, q_scale=0.05)
    v = torch.randn((400, 2, D), generator=torch.Generator().manual_seed(82)) * 2e4
    v[::7] = torch.sign(v[::7]) * 65468.5
    set_values(x, 0, v.clamp(-65468.5, 65468.5))
    assert x.v[0].abs().max() == 65468.5
    check_rows(x, Q.attn_paged(*x.args()))


@pytest.mark.parametrize("q_len", [3, 20, 200])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scores_that_vanish(Q, q_len, dtype):
    """Queries and scales so small that all scores are 0: the average of what a row sees."""
    for q_scale, scale in ((2.0 ** -100 if dtype == BF16 else 2.0 ** -14, 1e-20), (1.0, 1e-38), (1.0, 1e-44)):
        x = Batch([q_len], [q_len + 30], 4, 2, 64, 16, dtype, seed=83, q_scale=q_scale)
        check_rows(x, Q.attn_paged(*x.args(), scale=scale), scale=scale)


def test_bytes_that_hold_no_keys_do_not_count(Q):
    """Rows of a page behind the last key, whatever they hold, and blocks of zeros."""
    x = sharp([3, 1], [50, 70], 4, 2, 64, 16, F16, seed=76)
    for b, n in enumerate(x.kv_lens_host):
        v = x.v[b].float()
        v[:, :, 32:] = 0.0
        v[n // 2:, :, :32] *= 1e-3
        set_values(x, b, v)
    out = Q.attn_paged(*x.args())
    check_rows(x, out)
    assert (out[..., 32:] == 0).all()
