"""attn_paged with bounds that lie above the batch's lengths, as a server's caps do.

Tolerances: those of Batch.check."""

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_paged import BF16, F16, Batch, Q, clean_status, guarded   # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q_lens,heads,kv_heads,max_q", [
    ([1], 32, 8, 4),        # 4 rows per K/V head, bound 16
    ([1], 24, 8, 5),        # 3 and 15
    ([2], 32, 8, 3),        # 8 and 12
    ([1], 32, 8, 300),      # far above 16
    ([1], 8, 8, 1 << 40),
    ([1, 1], 8, 2, 4),      # 8 in two sequences
    ([5], 8, 8, 9),
    ([3, 1], 6, 6, 16),
])
def test_rows_bounded_loosely(Q, D, dtype, q_lens, heads, kv_heads, max_q):
    """Nothing is written beside a workspace of exactly the floats that the bounds ask for, and the result is that of
    the tight bound."""
    B = len(q_lens)
    x = Batch(q_lens, [20000 // B - 7 * b for b in range(B)], heads, kv_heads, D, 64, dtype, seed=61)
    total, max_kv = sum(q_lens), max(x.kv_lens_host)
    floats = Q.paged_workspace_floats(B, total, heads, kv_heads, max_q, max_kv, D)
    wide = Q.paged_workspace_floats(B, 16 * total, heads, kv_heads, max(1, 16 * kv_heads // heads), max_kv, D)
    assert 0 < floats <= wide
    raw = torch.full((floats + 2 * wide + 1024,), -77.0, device="cuda")   # room for any plan's states behind it
    out, out_raw, _ = guarded(x.q.shape, dtype)
    Q.attn_paged(*x.args()[:6], max_q, max_kv, out=out, workspace=raw[512:512 + floats])
    assert (raw[:512] == -77.0).all() and (raw[512 + floats:] == -77.0).all()
    assert (out_raw[:256] == 0x5A).all() and (out_raw[-256:] == 0x5A).all()
    x.check(out)
    tight = Q.attn_paged(*x.args())
    if max_q >= total:   # the same plan
        assert torch.equal(out, Q.attn_paged(*x.args()[:6], total, max_kv))
    x.check(tight)


def spread(n, low, high):
    """n lengths from low to high, far ones among them, in no order."""
    return [low + (high - low) * (i * i * 7919 % 101) // 100 for i in range(n)]


BATCHES = {
    # more sequences than are planned for on the device: shares by the bounds, one, two and three of them
    "70 bursts": ([5] * 70, spread(70, 5, 3000), 4, 1),
    "90 bursts of 1 to 6": ([1 + i % 6 for i in range(90)], spread(90, 6, 2500), 4, 1),
    "140 bursts": ([17] * 140, spread(140, 17, 1000), 1, 1),
    "70 with 2 chunks": ([1] * 30 + [300] + [2] * 20 + [129] + [1] * 18, [3000] + spread(69, 300, 2500), 2, 1),
    "100 with empty ones": ([(i % 4) * 7 for i in range(100)], [(i % 3) * 500 + 21 for i in range(100)], 2, 1),
    # more (row unit, K/V head) pairs than one wave of CTAs, so no shares: single tokens beside a chunk, a burst and a
    # long cache among them
    "63 tokens and a chunk": ([1] * 40 + [128] + [1] * 23, spread(63, 1, 900) + [2000], 32, 8),
    "one burst, a long cache": ([5] + [1] * 19, [400] * 9 + [20000] + [400] * 10, 32, 8),
    "160 chunks": ([150] * 20, spread(20, 150, 700), 8, 8),
    # 64 sequences exactly, planned on the device
    "64 bursts": ([6] * 64, spread(64, 6, 2000), 3, 1),
}


@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("loose", [False, True])
def test_batches_beyond_the_plans(Q, name, D, dtype, loose):
    q_lens, kv_lens, heads, kv_heads = BATCHES[name]
    if name == "63 tokens and a chunk":
        kv_lens = kv_lens[:40] + [2000] + kv_lens[40:63]
    x = Batch(q_lens, kv_lens, heads, kv_heads, D, 16, dtype, seed=62)
    max_q, max_kv = max(q_lens) + 3 * loose, max(kv_lens) + (16 if loose else 0)
    B, total = len(q_lens), sum(q_lens)
    floats = Q.paged_workspace_floats(B, total, heads, kv_heads, max_q, max_kv, D)
    ws, ws_raw, _ = guarded((max(floats, 4),), torch.float32)
    out, out_raw, _ = guarded(x.q.shape, dtype)
    Q.attn_paged(*x.args()[:6], max_q, max_kv, out=out, workspace=ws)
    x.check(out)
    for raw in (ws_raw, out_raw):
        assert (raw[:256] == 0x5A).all() and (raw[-256:] == 0x5A).all()
