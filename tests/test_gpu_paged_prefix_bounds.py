"""attn_paged_prefix with bounds made for long prefixes while the prefix on the device is short, or none: the launches for the own
keys find out there how many they are.

Tolerances: those of test_gpu_paged_range.py."""

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_paged import BF16, F16, Q, clean_status   # noqa: F401 (fixtures)
from tests.test_gpu_paged_range import Shared, before, check

pytestmark = pytest.mark.gpu


def is_shared(Q, x, args):
    """Whether the call shares the prefix: then what the sequences' own tables name for it is not read, else it is recorded."""
    assert Q.device_status(clear=True)[0] == Q.Q8A_OK and int(x.len) >= x.page
    table = args[3].clone()
    table[:, :int(x.len) // x.page] = 0x7FFFFFF0
    Q.attn_paged_prefix(*args[:3], table, *args[4:])
    return Q.device_status(clear=True)[0] == Q.Q8A_OK


OWN = [
    # new tokens, own keys, prefix, heads, kv heads: from own keys of less than a tile to the most that a cluster takes
    ([1] * 4, [1, 300, 2000, 7000], 3000, 8, 2),                        # clusters of eight, of which one to eight work
    ([1] * 40, [1 + 160 * i for i in range(40)], 900, 8, 2),            # of two
    ([4, 1, 2, 4], [4, 300, 2000, 7000], 3000, 8, 2),                   # 16 rows, clusters of four
    ([8, 1, 5, 8], [8, 100, 1000, 500], 3000, 8, 2),                    # 32 rows
    ([16, 3, 16, 1], [16, 60, 170, 100], 3000, 8, 2),                   # the tile kernel, in shares
    ([30] * 12, [30 + 11 * i for i in range(12)], 3000, 16, 8),
]


@pytest.mark.parametrize("q_lens,own,prefix,heads,kv_heads", OWN)
@pytest.mark.parametrize("D,dtype,page", [(64, F16, 16), (128, BF16, 64)])
def test_prefix_far_below_its_bound(Q, q_lens, own, prefix, heads, kv_heads, D, dtype, page):
    x = Shared(q_lens, own, prefix, heads, kv_heads, D, page, dtype, seed=sum(own))
    args = x.shared()
    assert is_shared(Q, x, args)
    for n in (prefix, 0, 64, prefix // 2, page - 1):
        x.len.fill_(n)
        out = Q.attn_paged_prefix(*args, out=torch.full_like(x.q, float("nan")))
        check(x, out, before(True), joined=True)
        assert torch.equal(out, Q.attn_paged_prefix(*args))


@pytest.mark.parametrize("q_len", [1, 4, 16])
def test_prefix_captured_for_any_length(Q, q_len):
    """One graph, replayed from a prefix of all keys but a few down to none and back."""
    x = Shared([q_len] * 4, [q_len, 200, 3000, 40], 4000, 8, 2, 128, 16, BF16, seed=q_len)
    args, out, graph = x.shared(), torch.empty_like(x.q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.attn_paged_prefix(*args, out=out)
    for n in (4000, 0, 1000, 15, 4000):
        x.len.fill_(n)
        x.q.normal_()
        out.fill_(float("nan"))
        graph.replay()
        check(x, out, before(True), joined=True)


def set_scale(x, pages, kept, b, key, bits, value, sequences):
    """Block 0 of row `key` of sequence b gets the scale of these bits; the sequences keep it as `value`."""
    slot = int(x.slots(b, torch.tensor([key], device="cuda")))
    block = pages[slot // x.page, :, slot % x.page, :34]
    block[:, 0], block[:, 1] = bits & 255, bits >> 8
    codes = block[:, 2:].contiguous().view(torch.int8).double().cpu()
    for s in sequences:
        kept[s] = torch.as_tensor(kept[s]).clone()
        kept[s][key, :, :32] = codes * value


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
def test_prefix_scales_beyond_fp16(Q, q_len, D, dtype):
    """Scales of V above 515.5, infinite and NaN: 515.5 in a prefix that is shared; as they are behind it, and in a call
    that does not share."""
    x = Shared([q_len] * 4, [300, 40, 100, 200], 640, 8, 2, D, 16, dtype, seed=q_len)
    every = range(4)
    set_scale(x, x.v_pages, x.v, 0, 100, 0x67D0, 515.5, every)         # 2000
    args = x.shared()
    assert is_shared(Q, x, args) and not is_shared(Q, x, (*x.args(), x.pages, x.len))
    check(x, Q.attn_paged_prefix(*args), before(True), joined=True)
    set_scale(x, x.v_pages, x.v, 1, 650, 0x6400, 1024.0, [1])          # sequence 1's own
    check(x, Q.attn_paged_prefix(*args), before(True), joined=True)
    set_scale(x, x.v_pages, x.v, 0, 100, 0x67D0, 2000.0, every)
    check(x, Q.attn_paged_prefix(*x.args(), x.pages, x.len), before(True), joined=True)
    for bits in (0x7C00, 0x7E00):
        set_scale(x, x.v_pages, x.v, 0, 100, bits, 515.5, every)
        check(x, Q.attn_paged_prefix(*args), before(True), joined=True)


@pytest.mark.parametrize("q_lens,own,prefix", [([1, 1, 1], [1, 1, 1], 16), ([1, 0, 1, 1], [1, 0, 33, 7], 40), ([2, 1, 3], [2, 90, 3], 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_smallest_shared_batches(Q, q_lens, own, prefix, causal):
    """One K/V head, one query head, few keys: a prefix of a page, with bounds long enough for it to be shared."""
    x = Shared(q_lens, own, prefix, 1, 1, 64, 16, F16, seed=len(q_lens))
    entries = (1 << 23) // 16
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((len(q_lens), entries + 8), 0x7FFFFFFF, **i32)
    table[:, :x.table.shape[1]] = x.table
    pages = torch.full((entries,), 0x7FFFFFFF, **i32)
    pages[:len(x.pages)] = x.pages
    args = x.q, x.k_pages, x.v_pages, table, x.kv_lens, x.cu_q, max(q_lens), entries * 16 + 100
    assert is_shared(Q, x, (*args, pages, x.len))
    check(x, Q.attn_paged_prefix(*args, pages, x.len, causal=causal), before(causal), joined=True)


@pytest.mark.parametrize("q_len", [1, 3, 6, 20])
@pytest.mark.parametrize("D", [64, 128])
def test_bound_of_all_keys(Q, q_len, D):
    """max_prefix = max_kv, as for prefixes of any length: one long sequence among short ones, nothing to all of it shared."""
    x = Shared([q_len] * 6, [q_len, 9000, 40, 300, 77, 21], 2000, 8, 2, D, 16, F16, seed=q_len)
    q, k_pages, v_pages, table, lens, cu, max_q, max_kv, pages, length = x.shared()
    args = q, k_pages, v_pages, table, lens, cu, max_q, pages.shape[0] * x.page, pages, length
    assert is_shared(Q, x, args)
    for n in (2000, 0, 1000, 16):
        x.len.fill_(n)
        check(x, Q.attn_paged_prefix(*args, out=torch.full_like(x.q, float("nan"))), before(True), joined=True)
