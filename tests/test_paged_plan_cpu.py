"""What attn_paged launches against the workspace it accepts, and which buffers of the paged calls may share memory (no
GPU needed): the library runs in a child process whose launches are replaced, so that every plan can be looked at
and nothing reaches a device."""

import ctypes
import itertools
import json
import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT

FIELDS = ("few_calls", "few_rows", "few_direct", "few_limit", "tiles_calls", "tiles_floats", "tiles_part", "shares", "share_tiles")
WORKSPACE = 0x7000000000   # never dereferenced


def child(cases):
    """Runs in the child: the launches of each case (total_q, heads, kv_heads, max_q, max_kv, D, batch, page)."""
    from chunked_prefill_attention_gb300 import q8attn as Q
    lib, rec = Q.load(), ctypes.CDLL(None)
    P = ctypes.c_void_p
    few_floats = lib["_ZN3q8a16paged_few_floatsEil"]
    few_floats.restype, few_floats.argtypes = ctypes.c_int64, [ctypes.c_int32, ctypes.c_int64]
    rec.record_start.argtypes, rec.record_take.argtypes = [P], [P]
    out = []
    for total, heads, kv, max_q, max_kv, D, batch, page in cases:
        floats = lib.q8a_paged_workspace_floats(batch, total, heads, kv, max_q, max_kv, D)
        width = -(-max_kv // page)
        rec.record_start(WORKSPACE)
        rc = lib.attn_paged(P(0x100000), 0, heads * D, total, heads, kv, D, P(0x200000), P(0x300000), 4, page,
                            kv * page * D // 32 * 34, P(0x400000), width, P(0x500000), P(0x600000), batch, max_q, max_kv,
                            0.125, 1, P(0x700000), P(WORKSPACE), floats, P(0))
        got = (ctypes.c_int64 * len(FIELDS))()
        rec.record_take(got)
        r = dict(zip(FIELDS, got), rc=rc, floats=floats)
        r["few_floats"] = few_floats(D, r["few_rows"]) if r["few_calls"] and not r["few_direct"] else 0
        out.append(r)
    print(json.dumps(out))


def child_overlap(cases):
    """Runs in the child: return codes and messages of calls named by (function, arguments)."""
    from chunked_prefill_attention_gb300 import q8attn as Q
    lib, out = Q.load(), []
    for name, args in cases:
        rc = getattr(lib, name)(*args)
        out.append((rc, lib.q8a_last_error().decode()))
    print(json.dumps(out))


@pytest.fixture(scope="module")
def launches(lib, tmp_path_factory):
    so = str(tmp_path_factory.mktemp("record") / "record.so")
    cuda = next((p for p in ("/usr/local/cuda/include", os.path.join(os.environ.get("CUDA_HOME", ""), "include"))
                 if os.path.exists(os.path.join(p, "cuda_runtime.h"))), None)
    if cuda is None:
        pytest.skip("no CUDA headers")
    r = subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", cuda, "-I", os.path.join(ROOT, "include"), "-o", so,
                        os.path.join(ROOT, "tests", "paged_launch_record.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases, name="child"):
        r = subprocess.run([sys.executable, "-c", f"import sys, json; from tests.test_paged_plan_cpu import {name}; "
                                                  f"{name}(json.load(sys.stdin))"],
                           cwd=ROOT, env=dict(os.environ, LD_PRELOAD=" ".join([os.environ.get("LD_PRELOAD", ""), so]).strip()),
                           input=json.dumps(cases), capture_output=True,
                           text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        return json.loads(r.stdout)

    return run


def check(case, r):
    assert r["rc"] == 0, (case, r)
    assert r["few_calls"] + r["tiles_calls"] > 0, (case, r)
    assert r["few_floats"] + r["tiles_floats"] <= r["floats"], (case, r)
    if r["tiles_calls"]:
        assert r["tiles_part"] >= r["few_floats"], (case, r)   # the two kernels' states lie apart


def test_workspace_holds_what_is_launched_whatever_the_bounds(launches):
    """max_q is a bound: above total_q the plan and the launch have to take it for the same number of rows."""
    cases = []
    for total, group, max_q, max_kv, D, batch in itertools.product(
            (1, 2, 3, 16, 40, 300), (1, 3, 4, 8), (1, 2, 4, 9, 16, 17, 300, 1 << 20, (1 << 62) + 1),
            (1, 512, 1025, 70000), (64, 128), (1, 2, 70)):
        cases.append((total, 2 * group, 2, max_q, max_kv, D, batch, 16))
    for case, r in zip(cases, launches(cases)):
        check(case, r)


@pytest.mark.parametrize("D", [64, 128])
def test_shares_of_the_longest_caches(launches, D):
    """max_kv may be anything that the table's rows hold, also more than a length (an int32) can be; calls of more than
    64 sequences share by it."""
    cases = [(total, 1, 1, 5 + total // batch, max_kv, D, batch, 4096)
             for batch, total in ((65, 1200), (90, 2000), (140, 3100)) for max_kv in (100000, 1 << 31, 1 << 36, 1 << 42, ((1 << 31) - 1) << 12)]
    keys = 96 if D == 64 else 64
    for case, r in zip(cases, launches(cases)):
        check(case, r)
        assert r["shares"]
        most = -(-min(case[4], (1 << 31) - 65536) // keys)
        assert most // 3 <= r["share_tiles"] <= most, (case, r)   # one to three parts of the longest possible length


def test_a_scale_that_is_no_number_in_base_2_is_refused(launches):
    """The kernels take scale * log2(e), which passes fp32's range before the scale does."""
    call = [1 << 24, 0, 64, 1, 1, 1, 64, 1 << 40, 1 << 41, 99, 16, 16 * 68, 0x4000, 99, 0x5000, 0x6000, 1, 1, 64, 0.0, 1, 1 << 25, 0,
            0, 0]
    cases = [("attn_paged", call[:19] + [s] + call[20:]) for s in (2.3e38, 2.4e38, 3.4e38, 1e-30)]
    assert [rc for rc, _ in launches(cases, "child_overlap")] == [0, -1, -1, 0]


def rows_meet(a, sa, na, b, sb, nb, wa, wb=None):
    """By every pair of rows."""
    wb = wa if wb is None else wb
    return any(a + i * sa < b + j * sb + wb and b + j * sb < a + i * sa + wa for i in range(na) for j in range(nb))


def test_buffers_that_share_memory_are_refused(launches):
    """Exactly those: slices of one fused buffer lie between each other without sharing a byte."""
    import random
    rng = random.Random(5)
    B = 1 << 24
    cases, want = [], []
    for _ in range(3000):   # attn_rope: rows of 64 fp16 values
        n = rng.choice((1, 2, 3, 9))
        sx, so = rng.choice((64, 65, 128, 192, 320)), rng.choice((64, 128, 192, 320))
        x, out = B, B + 2 * rng.randrange(-2000, 2000)
        if x == out:
            continue
        cases.append(("attn_rope", (x, out, 0, n, 1, 64, sx, so, 0x1000, 0x2000, 64, 0, 1.0, 0, 0)))
        want.append(rows_meet(x, 2 * sx, n, out, 2 * so, n, 128))
    for _ in range(1500):   # attn_paged: q against out and the workspace
        n, sq = rng.choice((1, 2, 5)), 8 * rng.choice((8, 9, 16, 40))
        q, out = B, B + 16 * rng.randrange(-200, 200)
        floats = 2 * (320 * 8 * (8 + 2 * 8 * (64 + 2)))   # more than the few-row kernel's 64-channel states
        ws = B + 16 * rng.choice((rng.randrange(-200, 200), 1 << 22))
        if q == out:
            continue
        cases.append(("attn_paged", (q, 0, sq, n, 1, 1, 64, 1 << 40, 1 << 41, 99, 16, 16 * 68, 0x4000, 99, 0x5000, 0x6000, 1,
                                     n, 1500, 0.125, 1, out, ws, floats, 0)))
        used = 320 * 8 * (8 + 2 * 8 * (64 + 2)) * 4
        want.append(rows_meet(q, 2 * sq, n, out, 128, n, 128) or rows_meet(q, 2 * sq, n, ws, 1, 1, 128, used) or
                    rows_meet(out, 128, n, ws, 1, 1, 128, used))
    need = 2 * 16 * 68
    for _ in range(1500):   # append: pools, also page by page in one buffer; read: its outputs
        n, stride = rng.choice((1, 2, 7)), 16 * rng.choice((need // 16, need // 16 + 1, need // 8, need // 4))
        k, v = B, B + 16 * rng.randrange(-1200, 1200)
        cases.append(("q8kv_append_paged", (0x1000, 0x2000, 0, 4, 2, 64, 128, 128, 0x3000, k, v, n, 16, stride, 0, 0, 0, 0, 1.0, 0)))
        want.append(rows_meet(k, stride, n, v, stride, n, need))
        t = rng.choice((1, 3, 40))
        cases.append(("q8kv_read_paged", (B << 8, B << 8, n, 16, stride, 0x3000, t, 2, 64, k, v, 2, 0)))
        want.append(rows_meet(k, 1, 1, v, 1, 1, t * 2 * 64 * 4))
    big = [("attn_rope", (B, B + 64, 2, 1 << 31, 1, 64, 1 << 32, 1 << 32, 0x1000, 0x2000, 64, 0, 1.0, 0, 0)),
           ("q8kv_append_paged", (0x1000, 0x2000, 0, 4, 2, 64, 128, 128, 0x3000, B, B + need, (1 << 31) - 1, 16, 1 << 40, 0, 0,
                                  0, 0, 1.0, 0))]   # sizes beyond the address space
    got = launches(cases + big, "child_overlap")
    assert sum(want) > 500 and len(want) - sum(want) > 500
    for case, w, (rc, msg) in zip(cases, want, got):
        assert (rc == -1 and "overlap" in msg) if w else rc == 0, (case, w, rc, msg)
    assert got[-2][0] == -1 and got[-1][0] == 0
