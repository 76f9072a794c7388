"""The paged calls as a process makes them: the first calls of all inside a capture, and several threads at once."""

import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")

from tests.conftest import ROOT
from tests.test_gpu_paged import BF16, F16, Batch, Q, clean_status, gen   # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def first_calls():
    """Runs in a child whose first calls of the library are captured: every kernel's set-up happens there."""
    from chunked_prefill_attention_gb300 import q8attn as Q
    g = torch.Generator(device="cuda").manual_seed(3)
    jobs = []
    for D in (64, 128):
        for q_lens, width, dtype in (([1], 8, F16), ([1, 2], 80, BF16), ([9], 40, F16), ([30, 20], 40, BF16), ([300], 20, F16),
                                     ([200, 1], 40, BF16)):
            T, B = sum(q_lens), len(q_lens)
            pages = [torch.zeros((B * width, 2, 64, Q.row_bytes(D)), dtype=torch.uint8, device="cuda") for _ in range(2)]
            keys = torch.randn((2, B * width * 64, 2, D), generator=g, device="cuda").to(dtype)
            pos = torch.arange(B * width * 64, device="cuda")
            x = torch.randn((T, 8, D), generator=g, device="cuda").to(dtype)
            floats = Q.paged_workspace_floats(B, T, 8, 2, max(q_lens), width * 64, D)
            jobs.append((x, keys, pages, pos, torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width),
                         torch.full((B,), width * 64 - 5, dtype=torch.int32, device="cuda"),
                         torch.tensor([0] + list(torch.tensor(q_lens).cumsum(0)), dtype=torch.int32, device="cuda"),
                         max(q_lens), width * 64, Q.rope_inv_freq(D, device="cuda"),
                         torch.empty(max(floats, 4), device="cuda"), torch.empty_like(x), torch.empty_like(x),
                         tuple(torch.empty_like(k) for k in keys)))

    def run():
        for i, (x, keys, pages, pos, table, lens, cu, max_q, max_kv, f, ws, turned, out, back) in enumerate(jobs):
            Q.attn_rope(x, pos[:len(x)], f, interleaved=bool(i & 1), out=turned)
            Q.q8kv_append_paged(keys[0], keys[1], *pages, pos, pos, f, interleaved=bool(i & 1))
            Q.q8kv_read_paged(*pages, pos, x.dtype, out=back)
            Q.attn_paged(turned, *pages, table, lens, cu, max_q, max_kv, out=out, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    got = [(j[-2].clone(), j[-1][0].clone(), j[2][0].clone()) for j in jobs]
    for j in jobs:
        for t in (j[-2], *j[-1], *j[2]):
            t.zero_()
    run()
    torch.cuda.synchronize()
    for (out, k, rows), j in zip(got, jobs):
        assert torch.equal(out, j[-2]) and torch.equal(k, j[-1][0]) and torch.equal(rows, j[2][0])
        assert out.abs().sum() > 0
    assert Q.device_status(clear=True) == (0, 0)
    print("same")


def test_the_first_calls_of_a_process_are_captured(Q):
    r = subprocess.run([sys.executable, "-c", "from tests.test_gpu_paged_process import first_calls; first_calls()"], cwd=ROOT,
                       env=dict(os.environ), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_threads(Q):
    """Four threads, each with a stream and a batch of its own, among them refused calls: results as alone, and each
    thread's own error text."""
    batches = [Batch([1, 2], [3000, 500], 8, 2, 128, 64, BF16, seed=91), Batch([300], [700], 4, 2, 64, 16, F16, seed=92),
               Batch([20, 3], [900, 4000], 4, 1, 64, 32, F16, seed=93), Batch([1], [300], 4, 4, 64, 16, F16, seed=94)]
    want = [Q.attn_paged(*x.args()) for x in batches]
    torch.cuda.synchronize()
    failures, start = [], threading.Barrier(len(batches))

    def work(i):
        x = batches[i]
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for n in range(40):
                    got = Q.attn_paged(*x.args())
                    try:
                        Q.attn_paged(*x.args()[:7], 1 << (30 + i))
                        failures.append("not refused")
                    except Q.Q8AttnError as e:
                        if str(1 << (30 + i)) not in str(e):
                            failures.append(str(e))
                    if n % 8 == 7 and not torch.equal(got, want[i]):
                        failures.append((i, n))
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001 (reported by the test)
            failures.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(batches))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[:3]
