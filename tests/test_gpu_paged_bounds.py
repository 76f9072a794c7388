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
