"""The attention in a window with sinks and behind a shared prefix, against a plain 64-bit implementation.

Tolerances: those of test_gpu_paged.py (its docstring derives them).  Behind a prefix the prefix's part comes from the
tile kernel whatever the rows' number, so its terms always count; and the two states are joined by their logarithms, each
off by 2^-24 of itself and by log2's 2^-23, at most 2^-24 (1.5 G + 32) + 2^-23 for up to 2^31 keys, so weights by less than
2^-23 G + 2^-18, in the numerator and the denominator.
"""

import math

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_paged import BF16, F16, Batch, clean_status, gen, unit   # noqa: F401  (a fixture among them)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q(lib):
    from chunked_prefill_attention_gb300 import q8attn
    yield q8attn
    torch.cuda.synchronize()


def check(x, out, visible, scale=None, sequences=None, joined=False):
    """Every row of every sequence; visible(positions [n_q, 1], keys [n]) says what a row sees."""
    scale = 1 / math.sqrt(x.D) if scale is None else scale
    u, row = unit(out.dtype), 0
    for b, (nq, n) in enumerate(zip(x.q_lens, x.kv_lens_host)):
        if nq == 0 or (sequences is not None and b not in sequences):
            row += nq
            continue
        q = x.q[row:row + nq].double()
        k, v = x.k[b].cuda(), x.v[b].cuda()
        seen = visible(torch.arange(nq, device="cuda")[:, None] + n - nq, torch.arange(n, device="cuda")[None])
        for h in range(q.shape[1]):
            kh = h // x.group
            s = q[:, h] @ k[:, kh].T * scale
            G = (q[:, h].abs() @ k[:, kh].abs().T * scale).amax() if n else 0.0
            p = torch.where(seen, s, -math.inf)
            top = p.amax(1, keepdim=True) if n else torch.zeros((nq, 1), device="cuda")
            p = torch.nan_to_num(torch.exp(p - torch.where(top == -math.inf, 0, top)), nan=0.0)
            total = p.sum(1, keepdim=True)
            p = p / torch.where(total == 0, 1, total)
            y, A = p @ v[:, kh], p @ v[:, kh].abs()
            got = out[row:row + nq, h].double()
            tol = (2.0 ** -11 * (1 if out.dtype == F16 else 2) + 2 * (2.0 ** -19 * G + 2.0 ** -21)) * A
            if joined:
                tol = tol + 2 * (2.0 ** -23 * G + 2.0 ** -18) * A
            if joined or nq * x.group > 64:
                tol = tol + 2.0 ** -11 * y.abs() + 2.0 ** -32 * (seen.double() @ v[:, kh].abs())
            tol = tol + u * (y.abs() + tol) + 2.0 ** -25
            bad = ~((got - y).abs() <= tol)
            assert not bad.any(), (b, h, int(bad.sum()), float((got - y).abs().max()), float(tol.max()))
        row += nq


# ------------------------------------------------------------------ window --


def in_window(window, sinks):
    return lambda p, j: (j <= p) & ((j > p - window) | (j < sinks))


WINDOW = [
    # new tokens, keys, heads, kv heads, D, page, window, sinks
    ([1], [1], 1, 1, 64, 16, 1, 0),
    ([1], [50], 4, 4, 64, 16, 1, 1),
    ([1], [1000], 8, 2, 64, 16, 100, 4),
    ([1], [5000], 32, 8, 128, 64, 1000, 4),
    ([1], [70001], 8, 8, 64, 128, 3001, 0),
    ([1], [20000], 4, 1, 128, 16, 19990, 40),
    ([1] * 5, [1, 700, 16, 0, 4097], 8, 2, 64, 16, 33, 2),
    ([1, 0, 1, 1], [300, 50, 17, 1000], 12, 4, 128, 32, 64, 16),
    ([2, 3, 1, 5], [2, 3, 900, 77], 4, 2, 64, 16, 7, 1),
    ([4], [3000], 8, 8, 128, 256, 5, 1500),
    ([16, 9], [1000, 9], 8, 2, 64, 64, 20, 33),
    ([1] * 300, [(37 * i) % 1900 for i in range(300)], 4, 4, 64, 16, 90, 5),
    ([5, 4], [3, 2], 2, 1, 64, 16, 2, 1),               # more new tokens than keys
    ([40], [40], 2, 2, 64, 16, 3, 0),
    ([64, 3], [5000, 3], 4, 2, 128, 16, 700, 70),
    ([128], [3000], 2, 2, 64, 32, 500, 3),
    ([300], [300], 4, 2, 64, 128, 1, 0),
    ([300], [9000], 4, 2, 64, 128, 129, 97),
    ([513], [1500], 4, 1, 128, 64, 96, 1),
    ([1025, 1, 77], [1025, 600, 2000], 4, 4, 64, 32, 200, 8),
    ([200, 333, 0, 65], [1000, 333, 10, 70], 6, 2, 128, 16, 64, 64),
    ([700], [700], 7, 1, 128, 32, 333, 0),
    ([2500], [2600], 3, 3, 64, 16, 1000, 4),
    ([50] * 70, [100 + 57 * i for i in range(70)], 2, 1, 64, 16, 400, 10),   # more sequences than are planned by length
    ([257], [4001], 3, 1, 64, 128, 1 << 40, 0),         # windows and sinks beyond any length
    ([9], [400], 8, 2, 128, 16, 3, 1 << 40),
]


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,D,page,window,sinks", WINDOW)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_window(Q, q_lens, kv_lens, heads, kv_heads, D, page, window, sinks, dtype):
    x = Batch(q_lens, kv_lens, heads, kv_heads, D, page, dtype, seed=len(q_lens) + sum(kv_lens))
    out = torch.full_like(x.q, float("nan"))
    got = Q.attn_paged_window(*x.args(), window, sinks, out=out)
    assert got.data_ptr() == out.data_ptr()
    check(x, got, in_window(window, sinks))
    if window > max(kv_lens):   # every key is in it
        x.check(got)


@pytest.mark.parametrize("q_len", [1, 6, 30, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_window_hides_whatever_is_behind_it(Q, q_len, D):
    """Keys and values of any scale, infinite and NaN among them, that no row of the window sees, between the sinks and
    the window: the pages there may have been given away."""
    window, sinks, n = 150, 20, 2000
    x = Batch([q_len, 1], [n, 900], 4, 2, D, 16, F16)
    for b, (nq, kv) in enumerate(zip(x.q_lens, x.kv_lens_host)):
        first = kv - nq - window + 1     # of the first row's window
        at = torch.arange(sinks, first, device="cuda")
        slots = x.slots(b, at)
        for pages in (x.k_pages, x.v_pages):
            rows = pages[slots // x.page, :, slots % x.page]
            blocks = rows.unflatten(-1, (-1, 34))
            blocks[::3, ..., 1], blocks[::3, ..., 0] = 0x7C, 0      # infinity
            blocks[1::3, ..., 1], blocks[1::3, ..., 0] = 0x7E, 1    # NaN
            blocks[2::3, ..., 1], blocks[2::3, ..., 0] = 0x7B, 0xFF  # 65504
            pages[slots // x.page, :, slots % x.page] = rows
        whole = torch.arange(-(-sinks // x.page), first // 32 * 32 // x.page, device="cuda")   # pages that nothing needs
        x.table[b, whole] = 0x7FFFFFF0
    check(x, Q.attn_paged_window(*x.args(), window, sinks), in_window(window, sinks))


@pytest.mark.parametrize("q_len", [3, 40])
@pytest.mark.parametrize("where", ["leaving", "entering"])
def test_window_keys_that_some_rows_see(Q, q_len, where):
    """A key of a very large value leaves the window between two rows, or enters with a later one: the rows that do not
    see it keep their results."""
    window, n = 50, 400
    x = Batch([q_len], [n], 4, 2, 64, 16, F16)
    want = Q.attn_paged_window(*x.args(), window, 2)
    key = n - q_len - window + 2 if where == "leaving" else n - q_len + 1   # rows 0 and 1 see it | all but row 0
    slot = int(x.slots(0, torch.tensor([key], device="cuda")))
    x.v_pages[slot // 16, :, slot % 16, 1] = 0x7C                  # an infinite scale of the first block
    x.v_pages[slot // 16, :, slot % 16, 0] = 0
    got = Q.attn_paged_window(*x.args(), window, 2)
    hidden = slice(2, None) if where == "leaving" else slice(0, 1)
    assert torch.isfinite(got[hidden]).all()
    assert (got[hidden] - want[hidden]).abs().max() <= 2.0 ** -9 * want.abs().max()   # sums in another order


def test_window_rows_pools_streams_and_repeats(Q):
    """Rows behind the last sequence stay, pools may be interleaved, a caller's workspace may hold anything, and the
    bits are the same every time, also on another stream."""
    for q_len, D in ((1, 64), (30, 128), (200, 64)):
        x = Batch([q_len, 2], [4000, 50], 8, 2, D, 32, F16, stray_rows=5, interleave_pools=True)
        out = torch.full_like(x.q, 9.0)
        Q.attn_paged_window(*x.args(), 700, 4, out=out)
        check(x, out, in_window(700, 4))
        assert (out[x.n_rows:] == 9.0).all()
        floats = Q.paged_window_workspace_floats(2, x.q.shape[0], 8, 2, max(q_len, 2), 4000, 700, 4, D)
        ws = torch.full((max(floats, 4),), float("nan"), device="cuda")
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(2):
                again = Q.attn_paged_window(*x.args(), 700, 4, out=torch.full_like(x.q, 9.0), workspace=ws)
        s.synchronize()
        assert torch.equal(out, again)


@pytest.mark.parametrize("q_len", [1, 40, 300])
def test_window_captured(Q, q_len):
    """Replayed as the sequences grow within their bounds."""
    x = Batch([q_len, q_len], [1800, 900], 8, 2, 64, 16, F16)
    out = torch.empty_like(x.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.attn_paged_window(*x.args(), 333, 5, out=out)
    full = x.kv_lens_host
    for cut in (0, 17, 400):
        x.kv_lens_host = [n - cut for n in full]
        x.kv_lens.copy_(torch.tensor(x.kv_lens_host))
        graph.replay()
        check_cut(x, out, 333, 5)


def check_cut(x, out, window, sinks):
    k, v = x.k, x.v
    x.k, x.v = ([t[:n] for t, n in zip(ts, x.kv_lens_host)] for ts in (k, v))
    check(x, out, in_window(window, sinks))
    x.k, x.v = k, v


def test_window_refusals(Q):
    x = Batch([1], [100], 4, 2, 64, 16, F16)
    Q.attn_paged_window(*x.args(), 10)
    for kw in (dict(window=0), dict(window=-5), dict(window=10, sinks=-1), dict(window=10, scale=0.0),
               dict(window=10, out=x.q), dict(window=10, workspace=torch.empty(0, device="cuda").half())):
        with pytest.raises(Q.Q8AttnError):
            Q.attn_paged_window(*x.args(), **kw)
    long = Batch([20], [5000], 4, 2, 64, 16, F16)
    with pytest.raises(Q.Q8AttnError):
        Q.attn_paged_window(*long.args(), 4000, workspace=torch.empty(64, device="cuda"))
    none = Q.attn_paged_window(x.q[:0], *x.args()[1:5], torch.zeros(2, dtype=torch.int32, device="cuda"), 1, 100, 10)
    assert none.shape == (0, 4, 64)


def test_window_bad_pages_are_recorded(Q):
    for q_len in (1, 200):
        x = Batch([q_len, q_len], [500, 300], 4, 2, 64, 16, F16)
        x.table[0, 30] = x.k_pages.shape[0]
        got = Q.attn_paged_window(*x.args(), 100, 4)
        assert Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG
        check(x, got, in_window(100, 4), sequences=[1])


# ------------------------------------------------------------------ prefix --


class Shared(Batch):
    """Sequences whose first `prefix` keys are the same; whole pages of them are the same pages."""

    def __init__(self, q_lens, own, prefix, heads, kv_heads, D, page, dtype, **kw):
        super().__init__(q_lens, [prefix + n for n in own], heads, kv_heads, D, page, dtype, **kw)
        self.prefix = prefix
        whole = prefix // page
        first = self.slots(0, torch.arange(prefix, device="cuda"))
        for b in range(1, len(q_lens)):
            slots = self.slots(b, torch.arange(prefix, device="cuda"))
            for pages in (self.k_pages, self.v_pages):
                pages[slots // page, :, slots % page] = pages[first // page, :, first % page]
            self.k[b][:prefix], self.v[b][:prefix] = self.k[0][:prefix], self.v[0][:prefix]
            self.table[b, :whole] = self.table[0, :whole]
        self.pages = self.table[0, :-(-prefix // page)].clone()
        self.len = torch.tensor([prefix], dtype=torch.int32, device="cuda")

    def shared(self, loose=True):
        """The call's arguments.  Whether the prefix is shared goes by the bounds; loose ones, as of a captured step made for
        long prefixes, make it so (but for two sequences of few rows, which never pay)."""
        if not loose:
            return (*self.args(), self.pages, self.len)
        q, k_pages, v_pages, table, lens, cu, max_q, max_kv = self.args()
        entries = (1 << 19) // self.page
        pages = torch.full((entries,), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
        pages[:len(self.pages)] = self.pages
        wide = torch.full((table.shape[0], entries + table.shape[1]), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        return q, k_pages, v_pages, wide, lens, cu, max_q, entries * self.page + max_kv - self.prefix, pages, self.len


def before(causal):
    return (lambda p, j: j <= p) if causal else (lambda p, j: j >= 0)


PREFIX = [
    # new tokens, own keys, prefix, heads, kv heads, D, page
    ([1, 1], [1, 1], 16, 1, 1, 64, 16),
    ([1, 1, 1], [1, 1, 1], 16, 1, 1, 64, 16),
    ([1, 1, 1], [1, 40, 7], 160, 8, 2, 64, 16),
    ([1, 1, 1], [1, 40, 7], 161, 8, 2, 64, 16),           # the prefix ends inside a page
    ([1] * 4, [9, 200, 30, 150], 2048, 32, 8, 64, 16),
    ([1] * 16, [50 + 31 * i for i in range(16)], 3000, 8, 2, 128, 64),
    ([1] * 70, [1 + 13 * i for i in range(70)], 777, 4, 1, 64, 32),
    ([1] * 300, [1 + i % 50 for i in range(300)], 1111, 4, 4, 64, 16),
    ([1, 1, 1], [3000, 5, 64], 96, 4, 4, 128, 32),
    ([2, 3, 1, 5], [2, 3, 900, 77], 500, 4, 2, 64, 16),
    ([4, 0, 4], [4, 0, 60], 6000, 16, 4, 128, 128),
    ([16, 9], [1000, 9], 400, 8, 2, 64, 64),
    ([30, 7, 25], [300, 7, 25], 1000, 8, 2, 128, 16),
    ([128, 1], [200, 1], 640, 2, 2, 64, 16),
    ([40] * 70, [40 + 9 * i for i in range(70)], 640, 3, 1, 64, 16),
    ([5] * 40, [5 + 11 * i for i in range(40)], 20000, 8, 2, 64, 256),
    ([2] * 5, [2] * 5, 5, 4, 2, 64, 16),                  # shorter than a page: nothing is shared
    ([200, 3], [200, 3], 300, 4, 2, 64, 16),              # as attn_paged
    ([7], [70], 300, 4, 2, 64, 16),
]


@pytest.mark.parametrize("q_lens,own,prefix,heads,kv_heads,D,page", PREFIX)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("loose", [True, False])
def test_prefix(Q, q_lens, own, prefix, heads, kv_heads, D, page, dtype, causal, loose):
    x = Shared(q_lens, own, prefix, heads, kv_heads, D, page, dtype, seed=len(q_lens) + sum(own))
    out = torch.full_like(x.q, float("nan"))
    Q.attn_paged_prefix(*x.shared(loose), causal=causal, out=out)
    check(x, out, before(causal), joined=True)


@pytest.mark.parametrize("q_len", [1, 20])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prefix_range_of_values(Q, q_len, D, dtype):
    """Sharp softmaxes, large and tiny values and queries."""
    for q_scale, v_scale, scale in [(12.0, 1.0, None), (1.0, 3000.0, None), (1.0, 2e-4, None), (2e-3, 1.0, 5.0)]:
        x = Shared([q_len] * 3, [300, 77, 20], 777, 4, 2, D, 16, dtype, seed=5, q_scale=q_scale, v_scale=v_scale)
        check(x, Q.attn_paged_prefix(*x.shared(), scale=scale), before(True), scale=scale, joined=True)


@pytest.mark.parametrize("q_len", [1, 12])
def test_prefix_of_any_length(Q, q_len):
    """The same batch with less of its prefix shared: nothing, part of a page, some pages; and with no bound given."""
    x = Shared([q_len] * 5, [400, 20, 33, 90, 250], 700, 8, 2, 64, 16, F16)
    for n in (0, 3, 16, 40, 333, 688, 700):
        x.len.fill_(n)
        check(x, Q.attn_paged_prefix(*x.shared()), before(True), joined=True)
    x.len.fill_(100)
    check(x, Q.attn_paged_prefix(*x.args(), x.table[1], x.len), before(True), joined=True)
    check(x, Q.attn_paged_prefix(*x.args(), x.table[1], x.len, max_prefix=0), before(True), joined=True)
    assert Q.device_status(clear=True)[0] == Q.Q8A_OK
    for n, most in ((300000, 200000), (-1, None), (-(1 << 31), None), ((1 << 31) - 1, None)):   # beyond the bound
        x.len.fill_(n)
        if n > 0:   # the keys up to the bound are taken: the prefix's own pages have to reach that far
            x.kv_lens.fill_(0)
            out = Q.attn_paged_prefix(*x.shared(), max_prefix=most)
            assert (out == 0).all()
            x.kv_lens.copy_(torch.tensor(x.kv_lens_host))
        else:
            check(x, Q.attn_paged_prefix(*x.shared(), max_prefix=most), before(True), joined=True)
        assert Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG


@pytest.mark.parametrize("q_len", [1, 3, 25])
def test_prefix_beyond_some_sequences(Q, q_len):
    """Sequences that are shorter than the prefix (padding of a captured step, a request that stops inside it) see what
    they have; one without keys gives 0."""
    x = Shared([q_len] * 4, [300, 20, 40, 100], 500, 8, 2, 64, 16, F16)
    for kv in ([800, 0, 200, 600], [800, 1, 499, 501], [2, 520, 300, 16]):
        x.kv_lens.copy_(torch.tensor(kv))
        full = x.kv_lens_host, x.k, x.v
        x.kv_lens_host = kv
        x.k, x.v = ([t[:n] for t, n in zip(ts, kv)] for ts in full[1:])
        x.kv_lens_host = full[0]
        out = Q.attn_paged_prefix(*x.shared())
        x.kv_lens_host = kv
        check(x, out, before(True), joined=True)
        x.kv_lens_host, x.k, x.v = full


def test_prefix_is_read_from_its_own_table(Q):
    """What the sequences' own tables name for the shared pages does not matter where the prefix is shared."""
    for q_len in (1, 30):
        x = Shared([q_len] * 4, [100, 40, 61, 33], 640, 8, 2, 64, 16, F16)
        want = Q.attn_paged_prefix(*x.shared())
        x.table[:, :640 // 16] = 0x7FFFFFF0
        assert torch.equal(want, Q.attn_paged_prefix(*x.shared()))   # and no index is recorded


def test_prefix_rows_streams_and_repeats(Q):
    """Rows before the first and behind the last sequence stay, and the bits are the same every time."""
    for q_len, dtype, D in ((1, F16, 64), (30, BF16, 128)):
        x = Shared([q_len] * 6, [500, 40, 61, 333, 70, 90], 2000, 8, 2, D, 32, dtype, stray_rows=5, interleave_pools=True)
        out = torch.full_like(x.q, 9.0)
        Q.attn_paged_prefix(*x.shared(), out=out)
        check(x, out, before(True), joined=True)
        assert (out[x.n_rows:] == 9.0).all()
        floats = Q.paged_prefix_workspace_floats(6, x.q.shape[0], 8, 2, q_len, x.shared()[7], 1 << 19, D)
        ws = torch.full((floats,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(2):
                again = Q.attn_paged_prefix(*x.shared(), out=torch.full_like(x.q, 9.0), workspace=ws)
        s.synchronize()
        assert torch.equal(out, again)
        with pytest.raises(Q.Q8AttnError):
            Q.attn_paged_prefix(*x.shared(), workspace=ws[:-8])
        x.cu_q[0] = 2                       # the first two rows belong to no sequence
        skipped = Q.attn_paged_prefix(*x.shared(), out=torch.full_like(x.q, 9.0))
        assert (skipped[:min(2, q_len)] == 9.0).all() if q_len > 1 else True
        Q.device_status(clear=True)


@pytest.mark.parametrize("q_len", [1, 20])
def test_prefix_captured(Q, q_len):
    """Replayed with other prefixes, lengths and queries."""
    x = Shared([q_len] * 5, [400, 20, 33, 90, 250], 900, 8, 2, 128, 16, BF16)
    out = torch.empty_like(x.q)
    graph = torch.cuda.CUDAGraph()
    args = x.shared()
    with torch.cuda.graph(graph):
        Q.attn_paged_prefix(*args, out=out)
    for n in (900, 64, 0, 560):
        x.len.fill_(n)
        x.q.normal_()
        graph.replay()
        check(x, out, before(True), joined=True)


def test_prefix_nan_and_infinite_queries_stay_in_their_rows(Q):
    for q_len in (1, 30):
        x = Shared([q_len] * 4, [300, 40, 50, 60], 2000, 4, 2, 64, 16, F16)
        want = Q.attn_paged_prefix(*x.shared())
        x.q[1, 0, 5] = float("nan")
        x.q[2, 3, 5] = float("inf")
        got = Q.attn_paged_prefix(*x.shared())
        touched = torch.zeros_like(got, dtype=torch.bool)
        touched[1, 0] = touched[2, 3] = True
        assert torch.isnan(got[1, 0]).all()
        assert torch.equal(got[~touched], want[~touched])


def test_prefix_refusals(Q):
    x = Shared([1] * 4, [30, 40, 60, 70], 100, 4, 2, 64, 16, F16)
    i32 = dict(dtype=torch.int32, device="cuda")
    Q.attn_paged_prefix(*x.shared())
    for table, length, kw in ((x.pages.long(), x.len, {}), (x.pages.cpu(), x.len, {}), (x.pages, x.len.long(), {}),
                              (x.pages, torch.zeros(2, **i32), {}), (x.pages, None, {}), (x.pages, x.len, dict(max_prefix=-1)),
                              (x.pages, x.len, dict(max_prefix=7 * 16 + 1)), (x.pages, x.len, dict(out=x.q)),
                              (x.pages[::2], x.len, {}), (x.pages, x.len, dict(scale=-1.0))):
        with pytest.raises(Q.Q8AttnError):
            Q.attn_paged_prefix(*x.args(), table, length, **kw)
    with pytest.raises(Q.Q8AttnError):
        Q.attn_paged_prefix(*x.shared(), workspace=torch.empty(8, device="cuda"))
    with pytest.raises(Q.Q8AttnError):
        Q.paged_prefix_workspace_floats(2, 2, 4, 2, 1, 100, -1)
    with pytest.raises(Q.Q8AttnError):
        Q.paged_window_workspace_floats(2, 2, 4, 2, 1, 100, 0, 0)


def test_prefix_bad_pages_are_recorded(Q):
    for q_len in (1, 30):
        x = Shared([q_len] * 3, [300, 40, 50], 320, 4, 2, 64, 16, F16)
        x.table[0, 30] = -1                  # one of the first sequence's own pages
        got = Q.attn_paged_prefix(*x.shared())
        assert Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG
        check(x, got, before(True), sequences=[1, 2], joined=True)
        x.table[0, 30] = x.table[0, 31]
        Q.attn_paged_prefix(*x.shared())
        assert Q.device_status(clear=True)[0] == Q.Q8A_OK
        x.pages[3] = x.k_pages.shape[0]
        Q.attn_paged_prefix(*x.shared())
        assert Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG


# ------------------------------------------------------------ used together --


@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
def test_a_server_of_these_calls(Q, D, dtype):
    """Prompts and then single tokens of several sequences: tables, norms with positions, pages, window; and behind the
    first sequence's prompt as a shared prefix, against plain attention on what the pages hold."""
    heads, kv, page, B, window, sinks = 8, 2, 16, 4, 60, 4
    g, f = gen(11), Q.rope_inv_freq(D, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    width, n_pages = 20, 100
    k_pages, v_pages = (torch.zeros((n_pages, kv, page, D // 32 * 34), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(n_pages, generator=g, device="cuda").int()
    n_free, lens = i32(n_pages), torch.zeros(B, dtype=torch.int32, device="cuda")
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2))
    x = Batch.__new__(Batch)
    x.group, x.D, x.page = heads // kv, D, page
    for new in ([90, 33, 150, 7], [1, 1, 1, 1], [1, 0, 3, 1], [20, 1, 1, 1]):
        total = sum(new) + 3
        lens, cu, slots, pos, n_free = Q.q8kv_extend_paged(i32(*new), lens, table, free, n_free, page, total)
        qkv = torch.randn((total, heads + 2 * kv, D), generator=g, device="cuda").to(dtype)
        q, k = Q.attn_norm_rope(qkv[:, :heads], qkv[:, heads:heads + kv], qw, kw, pos, f, out=(qkv[:, :heads], qkv[:, heads:heads + kv]))
        Q.q8kv_append_paged(k, qkv[:, heads + kv:], k_pages, v_pages, slots)
        x.q, x.q_lens, x.kv_lens_host = q, new, lens.tolist()
        x.k, x.v = [], []
        for b, n in enumerate(x.kv_lens_host):
            at = torch.arange(n, device="cuda")
            rows = Q.q8kv_read_paged(k_pages, v_pages, table[b, at // page].long() * page + at % page, torch.float32)
            x.k.append(rows[0].double())
            x.v.append(rows[1].double())
        args = (q, k_pages, v_pages, table, lens, cu, max(new), width * page)
        check(x, Q.attn_paged_window(*args, window, sinks), in_window(window, sinks))
        check(x, Q.attn_paged(*args), before(True))
    # the others go on from the first sequence's first 96 keys
    for b in range(1, B):
        table[b, :6] = table[0, :6]
        own = x.kv_lens_host[b]
        table[b, 6:8] = free[n_free - 2 * b:][:2] if own < 128 else table[b, 6:8]
        lens[b] = 100
    x.kv_lens_host, x.k, x.v, x.q_lens = lens.tolist(), [], [], [2, 1, 1, 2]
    for b, n in enumerate(x.kv_lens_host):
        at = torch.arange(n, device="cuda")
        rows = Q.q8kv_read_paged(k_pages, v_pages, table[b, at // page].long() * page + at % page, torch.float32)
        x.k.append(rows[0].double())
        x.v.append(rows[1].double())
    x.q = torch.randn((6, heads, D), generator=g, device="cuda").to(dtype)
    args = (x.q, k_pages, v_pages, torch.cat([table, torch.zeros((B, 1 << 15), dtype=torch.int32, device="cuda")], 1), lens,
            i32(0, 2, 3, 4, 6), 2, 1 << 19, torch.cat([table[0, :6], torch.zeros(1 << 15, dtype=torch.int32, device="cuda")]), i32(96))
    for max_prefix in (1 << 19, 96):   # shared, and not
        check(x, Q.attn_paged_prefix(*args, max_prefix=max_prefix), before(True), joined=True)
