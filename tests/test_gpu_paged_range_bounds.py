"""attn_paged_window and attn_paged_prefix with loose bounds, guarded buffers and random shapes, as a process makes the calls:
captured before anything else has run, from several threads, over pools beyond 4 GB, one call behind another.

Tolerances: those of test_gpu_paged_range.py."""

import os
import random
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")

from tests.conftest import ROOT
from tests.test_gpu_paged import BF16, F16, F32, Batch, Q, clean_status, gen, guarded   # noqa: F401 (fixtures)
from tests.test_gpu_paged_bounds import BATCHES
from tests.test_gpu_paged_range import Shared, before, check, in_window

pytestmark = pytest.mark.gpu


def guards_hold(*raws):
    return all((raw[:256] == 0x5A).all() and (raw[-256:] == 0x5A).all() for raw in raws)


@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("loose", [False, True])
def test_window_batches_beyond_the_plans(Q, name, D, dtype, loose):
    q_lens, kv_lens, heads, kv_heads = BATCHES[name]
    if name == "63 tokens and a chunk":
        kv_lens = kv_lens[:40] + [2000] + kv_lens[40:63]
    x = Batch(q_lens, kv_lens, heads, kv_heads, D, 16, dtype, seed=63)
    max_q, max_kv = max(q_lens) + 3 * loose, max(kv_lens) + (16 if loose else 0)
    B, total = len(q_lens), sum(q_lens)
    for window, sinks in ((700, 20), (1500, 0)):
        floats = Q.paged_window_workspace_floats(B, total, heads, kv_heads, max_q, max_kv, window, sinks, D)
        ws, ws_raw, _ = guarded((max(floats, 4),), torch.float32)
        out, out_raw, _ = guarded(x.q.shape, dtype)
        Q.attn_paged_window(*x.args()[:6], max_q, max_kv, window, sinks, out=out, workspace=ws)
        check(x, out, in_window(window, sinks))
        assert guards_hold(ws_raw, out_raw)


@pytest.mark.parametrize("seed", range(24))
def test_window_random(Q, seed):
    rng = random.Random(seed)
    D, kv_heads, group, page = rng.choice((64, 128)), rng.choice((1, 2, 3)), rng.choice((1, 2, 3, 4, 8)), rng.choice((16, 32, 64, 256))
    kind = rng.choice(("decode", "burst", "mixed", "prompts"))
    B = rng.randint(1, 9)
    q_lens = {"decode": [1] * B, "burst": [rng.randint(1, 24) for _ in range(B)],
              "mixed": [rng.choice((0, 1, 1, 3, 150)) for _ in range(B)], "prompts": [rng.randint(30, 700) for _ in range(B)]}[kind]
    kv_lens = [max(0, n + rng.choice((0, 0, 1, rng.randint(0, 300), rng.randint(0, 9000), -1))) for n in q_lens]
    dtype = rng.choice((F16, BF16))
    x = Batch(q_lens, kv_lens, kv_heads * group, kv_heads, D, page, dtype, seed=seed, interleave_pools=seed % 2 == 0, stray_rows=seed % 3)
    max_q, max_kv = max(max(q_lens), 1) + rng.choice((0, 0, 1, 40)), max(kv_lens) + rng.choice((0, page))
    window, sinks = rng.choice((1, 17, 64, 200, rng.randint(1, 6000))), rng.choice((0, 0, 1, 4, 33, rng.randint(0, 600)))
    floats = Q.paged_window_workspace_floats(len(q_lens), x.q.shape[0], kv_heads * group, kv_heads, max_q, max_kv, window, sinks, D)
    ws, ws_raw, _ = guarded((max(floats, 4),), torch.float32)
    out, out_raw, _ = guarded(x.q.shape, dtype)
    out.fill_(3.0)
    Q.attn_paged_window(*x.args()[:6], max_q, max_kv, window, sinks, out=out, workspace=ws)
    check(x, out, in_window(window, sinks))
    assert guards_hold(ws_raw, out_raw) and (out[x.n_rows:] == 3.0).all()


@pytest.mark.parametrize("seed", range(24))
def test_prefix_random(Q, seed):
    rng = random.Random(1000 + seed)
    D, kv_heads, group, page = rng.choice((64, 128)), rng.choice((1, 2, 3)), rng.choice((1, 2, 3, 4, 8)), rng.choice((16, 32, 64, 256))
    B = rng.choice((3, 5, 16, 66))
    q_lens = [1] * B if rng.random() < 0.5 else [rng.randint(0, rng.choice((3, 16, 128 // group))) for _ in range(B)]
    q_lens[-1] = max(1, q_lens[-1])
    own = [n + rng.choice((0, 0, 5, rng.randint(0, 200), rng.randint(0, 2000))) for n in q_lens]
    prefix, dtype, causal = rng.randint(1, 3000), rng.choice((F16, BF16)), rng.random() < 0.7
    x = Shared(q_lens, own, prefix, kv_heads * group, kv_heads, D, page, dtype, seed=seed, interleave_pools=seed % 2 == 0,
               stray_rows=seed % 3)
    args = list(x.shared(loose=seed % 4 != 3))
    args[6] += rng.choice((0, 0, 1)) if max(q_lens) * group < 120 else 0
    most = args[8].shape[0] * page
    floats = Q.paged_prefix_workspace_floats(B, x.q.shape[0], kv_heads * group, kv_heads, args[6], args[7], most, D)
    ws, ws_raw, _ = guarded((max(floats, 4),), torch.float32)
    out, out_raw, _ = guarded(x.q.shape, dtype)
    out.fill_(3.0)
    Q.attn_paged_prefix(*args, causal=causal, out=out, workspace=ws)
    check(x, out, before(causal), joined=True)
    assert guards_hold(ws_raw, out_raw) and (out[x.n_rows:] == 3.0).all()


@pytest.mark.parametrize("q_lens,kv,window", [([1], 9000, 5000), ([1, 1, 1], 20000, 4000), ([2, 1], 3000, 2047), ([1] * 20, 3000, 2500)])
@pytest.mark.parametrize("D", [64, 128])
def test_window_clusters_captured_and_shared_workspace(Q, q_lens, kv, window, D):
    """Calls that several CTAs of a cluster take, captured twice over one workspace and replayed in turn."""
    xs = [Batch(q_lens, [kv - 100 * b for b in range(len(q_lens))], 8, 2, D, 32, F16, seed=s) for s in (31, 32)]
    outs, graphs = [torch.zeros_like(x.q) for x in xs], []
    ws = torch.empty(max(4, Q.paged_window_workspace_floats(len(q_lens), xs[0].n_rows, 8, 2, max(q_lens), kv, window, 6, D)), device="cuda")
    for x, out in zip(xs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            Q.attn_paged_window(*x.args(), window, 6, out=out, workspace=ws)
        graphs.append(graph)
    for _ in range(2):
        for out in outs:
            out.fill_(float("nan"))
        graphs[0].replay()
        graphs[1].replay()
        for x, out in zip(xs, outs):
            check(x, out, in_window(window, 6))


def test_prefix_graphs_share_a_workspace(Q):
    for q_len in (1, 20):
        xs = [Shared([q_len] * 6, [q_len + 90 * i for i in range(6)], 900 + 50 * s, 8, 2, 64, 16, BF16, seed=s) for s in (1, 2)]
        floats = max(Q.paged_prefix_workspace_floats(6, x.n_rows, 8, 2, q_len, x.shared()[7], 1 << 19, 64) for x in xs)
        ws, outs, graphs, keep = torch.empty(floats, device="cuda"), [torch.zeros_like(x.q) for x in xs], [], []
        for x, out in zip(xs, outs):
            keep.append(x.shared())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                Q.attn_paged_prefix(*keep[-1], out=out, workspace=ws)
            graphs.append(graph)
        for _ in range(2):
            graphs[0].replay()
            graphs[1].replay()
            for x, out in zip(xs, outs):
                check(x, out, before(True), joined=True)


def test_window_and_prefix_offsets_beyond_32_bits(Q):
    """Pages whose byte offsets pass 2^32 (the pools are 5.7 GB each)."""
    D, HK, page, n_pages = 128, 8, 256, 20500
    kp = torch.zeros((n_pages, HK, page, 136), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    g = gen(52)
    at = torch.tensor([n_pages - 1, 3, n_pages - 2, 9, n_pages - 5], dtype=torch.int32, device="cuda")
    n = 1200
    k, v = (torch.randn((n, HK, D), generator=g, device="cuda").half() for _ in range(2))
    pos = torch.arange(n, device="cuda")
    slots = at[pos // page].long() * page + pos % page
    Q.q8kv_append_paged(k, v, kp, vp, slots)
    k2, v2 = Q.q8kv_read_paged(kp, vp, slots, F32)
    i32 = dict(dtype=torch.int32, device="cuda")
    for q_len in (1, 30, 300):
        x = Batch.__new__(Batch)
        x.group, x.D, x.page, x.q_lens, x.kv_lens_host = 2, D, page, [q_len], [n]
        x.q = torch.randn((q_len, 2 * HK, D), generator=g, device="cuda").half()
        x.k, x.v = [k2.double()], [v2.double()]
        args = (x.q, kp, vp, at[None], torch.tensor([n], **i32), torch.tensor([0, q_len], **i32), q_len, n)
        check(x, Q.attn_paged_window(*args, 500, 100), in_window(500, 100))
        if q_len == 300:
            continue
        x.q_lens, x.kv_lens_host, x.k, x.v = [q_len] * 4, [n] * 4, x.k * 4, x.v * 4
        x.q = torch.randn((4 * q_len, 2 * HK, D), generator=g, device="cuda").half()
        wide = torch.cat([at, torch.zeros(1 << 13, **i32)])
        check(x, Q.attn_paged_prefix(x.q, kp, vp, wide.repeat(4, 1), torch.full((4,), n, **i32),
                                     torch.arange(0, 4 * q_len + 1, q_len, **i32), q_len, 1 << 21, wide, torch.tensor([1000], **i32)),
              before(True), joined=True)


def chain(Q, steps, captured):
    """A server's step over and over, each call on what the one before it wrote; the caches and the outputs of all steps."""
    B, heads, kv, D, page, window, sinks = 5, 8, 2, 64, 16, 40, 3
    g = gen(7)
    i32 = dict(dtype=torch.int32, device="cuda")
    total, width, n_pages = B * 3, 40, 150
    pages = [torch.zeros((n_pages, kv, page, 68), dtype=torch.uint8, device="cuda") for _ in range(2)]
    table, free = torch.full((B, width), -1, **i32), torch.randperm(n_pages, generator=g, device="cuda").int()
    lens, n_free, new = torch.zeros(B, **i32), torch.tensor([n_pages], **i32), torch.zeros(B, **i32)
    out = (lens, torch.empty(B + 1, **i32), *(torch.empty(total, dtype=torch.int64, device="cuda") for _ in range(2)), n_free)
    qkv = torch.empty((total, heads + 2 * kv, D), dtype=F16, device="cuda")
    q, k, v = qkv.split([heads, kv, kv], 1)
    w, f = torch.ones(D, dtype=F16, device="cuda"), Q.rope_inv_freq(D, device="cuda")
    outs = [torch.zeros((total, heads, D), dtype=F16, device="cuda") for _ in range(2)]
    floats = max(Q.paged_window_workspace_floats(B, total, heads, kv, 3, width * page, window, sinks, D),
                 Q.paged_workspace_floats(B, total, heads, kv, 3, width * page, D), 4)
    ws = torch.empty(floats, device="cuda")

    def step():
        _, cu, slots, pos, _ = Q.q8kv_extend_paged(new, lens, table, free, n_free, page, total, out=out)
        Q.attn_norm_rope(q, k, w, w, pos, f, out=(q, k))
        Q.q8kv_append_paged(k, v, *pages, slots)
        Q.attn_paged_window(q, *pages, table, lens, cu, 3, width * page, window, sinks, out=outs[0], workspace=ws)
        Q.attn_paged(q, *pages, table, lens, cu, 3, width * page, out=outs[1], workspace=ws)

    inputs = [torch.randn(qkv.shape, generator=g, device="cuda").half() for _ in range(steps)]
    news = [torch.randint(0, 4, (B,), generator=g, device="cuda").int() for _ in range(steps)]
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    got = []
    torch.cuda.synchronize()
    for x, n in zip(inputs, news):
        qkv.copy_(x)
        new.copy_(n)
        graph.replay() if captured else step()
        got.append((outs[0].clone(), outs[1].clone(), lens.clone()))
    torch.cuda.synchronize()
    return got, pages, table


def test_steps_in_a_row(Q):
    """Without a wait of the host between the calls, and as a replayed graph: the same bits as with a wait behind every call."""
    real, waits = Q._call, []

    def waiting(*a):
        real(*a)
        torch.cuda.synchronize()
        waits.append(1)

    Q._call = waiting
    try:
        want, pages, table = chain(Q, 25, False)
    finally:
        Q._call = real
    assert len(waits) == 125
    for captured in (False, True):
        got, pages2, table2 = chain(Q, 25, captured)
        assert torch.equal(table, table2) and all(torch.equal(a, b) for a, b in zip(pages, pages2))
        for i, (a, b) in enumerate(zip(want, got)):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), i
    assert want[-1][0].abs().sum() > 0


def first_calls():
    """Runs in a child whose first calls of the library are captured: every kernel's set-up happens there."""
    from chunked_prefill_attention_gb300 import q8attn as Q
    got, pages, table = chain(Q, 4, True)
    xs, graphs, outs = [], [], []
    for D, dtype in ((64, F16), (128, BF16)):
        for q_len in (1, 3, 25, 200):
            xs.append(Shared([q_len] * 4, [q_len + 50 * i for i in range(4)], 3000, 8, 2, D, 32, dtype, seed=q_len))
    calls = []
    for x in xs:
        args, out = x.shared(), [torch.empty_like(x.q) for _ in range(2)]
        ws = torch.empty(max(4, Q.paged_prefix_workspace_floats(4, x.n_rows, 8, 2, max(x.q_lens), args[7], 1 << 19, x.D),
                             Q.paged_window_workspace_floats(4, x.n_rows, 8, 2, max(x.q_lens), max(x.kv_lens_host), 2500, 4, x.D)), device="cuda")
        calls.append((args, out, ws))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, (args, out, ws) in zip(xs, calls):
            Q.attn_paged_prefix(*args, out=out[0], workspace=ws)
            Q.attn_paged_window(*x.args(), 2500, 4, out=out[1], workspace=ws)
    graph.replay()
    for x, (args, out, ws) in zip(xs, calls):
        check(x, out[0], before(True), joined=True)
        check(x, out[1], in_window(2500, 4))
    assert Q.device_status(clear=True) == (0, 0)
    print("right")


def test_the_first_calls_of_a_process_are_captured(Q):
    r = subprocess.run([sys.executable, "-c", "from tests.test_gpu_paged_range_bounds import first_calls; first_calls()"], cwd=ROOT,
                       env=dict(os.environ), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "right" in r.stdout, r.stdout + r.stderr


def test_threads(Q):
    """Four threads, each with a stream and calls of its own, among them refused ones: results as alone."""
    xs = [Batch([1, 2], [9000, 500], 8, 2, 128, 64, BF16, seed=91), Batch([300], [700], 4, 2, 64, 16, F16, seed=92),
          Shared([1] * 5, [90, 40, 30, 20, 200], 2000, 8, 2, 64, 32, F16, seed=93),
          Shared([9] * 4, [90, 40, 30, 20], 2000, 8, 2, 128, 32, BF16, seed=94)]
    args = [x.shared() if isinstance(x, Shared) else x.args() for x in xs]
    call = lambda i: (Q.attn_paged_prefix(*args[i]) if isinstance(xs[i], Shared) else Q.attn_paged_window(*args[i], 4000, 4))
    want = [call(i) for i in range(4)]
    torch.cuda.synchronize()
    failures, start = [], threading.Barrier(4)

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for n in range(40):
                    got = call(i)
                    try:
                        Q.attn_paged_window(*xs[i].args(), -100 - i)
                        failures.append("not refused")
                    except Q.Q8AttnError as e:
                        if str(-100 - i) not in str(e) and "invalid sizes" not in str(e):
                            failures.append(str(e))
                    if n % 8 == 7 and not torch.equal(got, want[i]):
                        failures.append((i, n))
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001 (reported by the test)
            failures.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[:3]
