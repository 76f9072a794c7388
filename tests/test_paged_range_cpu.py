"""attn_paged_window and attn_paged_prefix on the host (no GPU needed): bad arguments are refused before any CUDA call; what
they launch fits the workspace they ask for, whatever the bounds; and the bound of a window's key tiles holds for every unit.
The launches run in a child process where they are replaced."""

import ctypes
import itertools
import json
import os
import random
import subprocess
import sys

import pytest

from tests.conftest import ROOT

FIELDS = ("kind", "mode", "part", "rows", "direct", "pair", "shares", "share_tiles", "ctas", "floats", "batch", "seqs", "window",
          "sinks", "state", "most", "join")
PLAIN, WINDOW, OWN, PREFIX = range(4)
WORKSPACE = 0x7000000000   # never dereferenced
P = ctypes.c_void_p


def child(cases):
    """Runs in the child: (call, arguments) each, the launches of it."""
    from chunked_prefill_attention_gb300 import q8attn as Q
    lib, rec = Q.load(), ctypes.CDLL(None)
    few_floats = lib["_ZN3q8a16paged_few_floatsEil"]
    few_floats.restype, few_floats.argtypes = ctypes.c_int64, [ctypes.c_int32, ctypes.c_int64]
    rec.record_start.argtypes, rec.record_take.argtypes = [P], [P]
    out = []
    for call, total, heads, kv, max_q, max_kv, D, batch, page, x, y in cases:
        width = -(-max_kv // page)
        head = (P(1 << 36), 0, heads * D, total, heads, kv, D, P(0x200000), P(0x300000), 4, page, kv * page * D // 32 * 34,
                P(0x400000), width, P(0x500000), P(0x600000), batch, max_q, max_kv)
        rec.record_start(WORKSPACE)
        if call == "window":
            floats = lib.q8a_paged_window_workspace_floats(batch, total, heads, kv, max_q, max_kv, x, y, D)
            rc = lib.attn_paged_window(*head, x, y, 0.125, P(1 << 38), P(WORKSPACE), floats, P(0))
        else:
            floats = lib.q8a_paged_prefix_workspace_floats(batch, total, heads, kv, max_q, max_kv, x, D)
            rc = lib.attn_paged_prefix(*head, P(0x800000), -(-x // page), P(0x900000), x, 0.125, y, P(1 << 38), P(WORKSPACE),
                                       floats, P(0))
        got = (ctypes.c_int64 * (8 * len(FIELDS)))()
        n = rec.record_take(got)
        launches = [dict(zip(FIELDS, got[len(FIELDS) * i:])) for i in range(n)]
        for a in launches:
            a["few_floats"] = few_floats(D, a["rows"]) if a["kind"] == 0 and not a["direct"] else 0
        out.append(dict(rc=rc, floats=floats, launches=launches))
    print(json.dumps(out))


@pytest.fixture(scope="module")
def launches(lib, tmp_path_factory):
    so = str(tmp_path_factory.mktemp("record") / "record.so")
    cuda = next((p for p in ("/usr/local/cuda/include", os.path.join(os.environ.get("CUDA_HOME", ""), "include"))
                 if os.path.exists(os.path.join(p, "cuda_runtime.h"))), None)
    if cuda is None:
        pytest.skip("no CUDA headers")
    r = subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", cuda, "-I", os.path.join(ROOT, "include"), "-o", so,
                        os.path.join(ROOT, "tests", "paged_range_record.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases):
        r = subprocess.run([sys.executable, "-c", "import sys, json; from tests.test_paged_range_cpu import child; "
                                                  "child(json.load(sys.stdin))"],
                           cwd=ROOT, env=dict(os.environ, LD_PRELOAD=" ".join([os.environ.get("LD_PRELOAD", ""), so]).strip()),
                           input=json.dumps(cases), capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        return json.loads(r.stdout)

    return run


def states_of(a, D):
    """Floats that a launch writes behind its `part`."""
    if a["kind"] == 0:
        return a["few_floats"]
    return a["ctas"] * 256 * (D + 2) if a["pair"] or a["shares"] or a["mode"] == PREFIX else 0


def test_window_launches_fit_their_workspace(launches):
    cases = [("window", total, 2 * group, 2, max_q, max_kv, D, batch, 16, window, sinks)
             for total, group, max_q, max_kv, D, batch, (window, sinks) in itertools.product(
                 (1, 2, 16, 300), (1, 4), (1, 4, 17, 300, (1 << 62) + 1), (1, 1025, 70000), (64, 128), (1, 2, 70),
                 ((1, 0), (100, 4), (5000, 0), (1 << 62, 1 << 62)))]
    for case, r in zip(cases, launches(cases)):
        D = case[6]
        assert r["rc"] == 0 and r["launches"], (case, r)
        used = []
        for a in r["launches"]:
            assert a["mode"] == WINDOW and a["window"] == min(case[9], 0x7FFF0000) and a["sinks"] == min(case[10], 0x7FFF0000)
            used.append((a["part"], a["part"] + states_of(a, D)))
        for lo, hi in used:
            assert 0 <= lo and hi <= r["floats"], (case, r)
        if len(used) == 2:   # the two kernels' states lie apart
            assert used[1][1] <= used[0][0] or used[0][1] <= used[1][0]


def test_prefix_launches_fit_their_workspace(launches):
    cases = [("prefix", total, 2 * group, 2, max_q, max_kv, D, batch, 16, most, causal)
             for total, group, max_q, max_kv, D, batch, most, causal in itertools.product(
                 (1, 3, 40, 300), (1, 4, 8), (1, 2, 5, 30, 300, (1 << 62) + 1), (1, 700, 70000, 3000000), (64, 128), (1, 3, 70, 300),
                 (0, 16, 65536, 2500000), (0, 1))]
    shared = 0
    for case, r in zip(cases, launches(cases)):
        _, total, heads, kv, max_q, max_kv, D, batch, page, most, causal = case
        assert r["rc"] == 0 and r["launches"], (case, r)
        modes = [a["mode"] for a in r["launches"]]
        if PREFIX not in modes:
            assert set(modes) == {PLAIN} or (modes == [WINDOW] and r["launches"][0]["window"] == 0x7FFF0000)
            for a in r["launches"]:
                assert a["part"] + states_of(a, D) <= r["floats"]
            continue
        shared += 1
        assert modes == [OWN, PREFIX]
        own, prefix = r["launches"]
        assert min(max_q, total) * heads // kv <= 128 and batch > 1
        for a in (own, prefix):   # behind the rows' states, which both use
            assert a["state"] == 0 and a["part"] >= total * heads * (D + 1) and a["part"] % 4 == 0
            assert a["part"] + states_of(a, D) <= r["floats"], (case, a)
            assert a["most"] == most
        assert (own["batch"], prefix["batch"], prefix["seqs"]) == (batch, 1, batch)
        assert prefix["join"] in (1, 8)
        assert prefix["share_tiles"] == (0 if prefix["shares"] else 0x3FFFFFFF)
        assert own["kind"] == 0 or own["pair"]
    assert shared > 200


def test_the_rule_of_sharing(launches):
    """Long prefixes and many sequences share, short ones and few do not; so does a call whose sequences fill the tiles."""
    def is_shared(batch, rows, prefix, kv=8, group=4, D=128):
        r = launches([("prefix", batch * rows, kv * group, kv, rows, prefix + 500, D, batch, 64, prefix, 1)])[0]
        assert r["rc"] == 0, r
        return any(a["mode"] == PREFIX for a in r["launches"])
    assert is_shared(64, 1, 32768) and is_shared(16, 4, 8192) and is_shared(64, 1, 32768, kv=1)
    assert not is_shared(1, 1, 1 << 20) and not is_shared(2, 1, 1 << 20) and not is_shared(64, 1, 64)
    assert not is_shared(64, 33, 32768) and is_shared(64, 32, 32768)
    assert is_shared(1 << 20, 1, 1 << 30, kv=64, group=1)   # no overflow on the way


def test_window_tiles_bound_every_unit(lib):
    """The most tiles that any unit of 128 or 256 rows of a sequence takes, computed unit by unit, against the bound that the
    shares are planned by."""
    bound = lib["_ZN3q8a12window_tilesElllibi"]
    bound.restype, bound.argtypes = ctypes.c_int64, [ctypes.c_int64] * 3 + [ctypes.c_int32, ctypes.c_bool, ctypes.c_int32]
    rng = random.Random(3)
    for _ in range(4000):
        D, pair, group = rng.choice((64, 128)), rng.random() < 0.5, rng.choice((1, 2, 3, 4, 7, 8, 16))
        bn, per, piece = (96 if D == 64 else 64), (128 if pair else 256), rng.choice((16, 32))
        n_q = rng.choice((1, 5, 40, 300, 1000))
        kv = max(0, n_q + rng.choice((-3, 0, 1, 50, 500, 3000)))
        window, sinks = rng.choice((1, 2, 31, 64, 97, 500, 5000)), rng.choice((0, 1, 16, 64, 97, 200, 4000))
        for r0 in range(0, n_q * group, per):
            first, last = r0 // group, min(r0 + per - 1, n_q * group - 1) // group
            end = max(0, min(kv, kv - n_q + last + 1))
            low = max(0, kv - n_q + first - window + 1)
            base, sink = low // piece * piece, -(-min(sinks, end) // bn)
            if sink * bn >= base:
                sink = base = 0
            assert sink + -(-max(end - base, 0) // bn) <= bound(kv, window, sinks, group, pair, D)


def test_window_and_prefix_refusals(lib):
    from chunked_prefill_attention_gb300 import q8attn as Q
    A = [P(0x10000000 * (i + 1)) for i in range(10)]
    bad, mis, uns = Q.Q8A_ERR_INVALID_ARG, Q.Q8A_ERR_MISALIGNED, Q.Q8A_ERR_UNSUPPORTED
    base = dict(q=A[0], dtype=0, stride=512, total=3, heads=8, kv=2, D=64, k=A[1], v=A[2], pages=4, page=16, ps=2 * 16 * 68, table=A[3],
                width=20, lens=A[4], cu=A[5], batch=3, max_q=1, max_kv=300)

    def head(kw):
        d = {**base, **{k: v for k, v in kw.items() if k in base}}
        return list(d.values())

    def window(window=100, sinks=4, scale=0.125, out=A[6], ws=A[7], floats=1 << 24, **kw):
        return lib.attn_paged_window(*head(kw), window, sinks, scale, out, ws, floats, P(0))

    def prefix(ptab=A[8], entries=10, plen=A[9], most=160, scale=0.125, out=A[6], ws=A[7], floats=1 << 24, **kw):
        return lib.attn_paged_prefix(*head(kw), ptab, entries, plen, most, scale, 1, out, ws, floats, P(0))

    for call, name in ((window, "attn_paged_window"), (prefix, "attn_paged_prefix")):
        for kw in (dict(heads=0), dict(heads=7), dict(kv=0), dict(batch=-1), dict(batch=(1 << 20) + 1), dict(total=-1), dict(total=1 << 31),
                   dict(max_q=-1), dict(max_kv=-1), dict(max_kv=321), dict(stride=511), dict(scale=0.0), dict(scale=float("nan")),
                   dict(scale=3e38), dict(pages=0), dict(page=24), dict(ps=100), dict(k=P(0)), dict(q=P(0)), dict(out=P(0)),
                   dict(lens=P(0)), dict(cu=P(0)), dict(table=P(0)), dict(out=A[0]), dict(width=-1)):
            assert call(**kw) == bad, (name, kw)
            assert name in lib.q8a_last_error().decode()
        for kw in (dict(D=96), dict(dtype=2)):
            assert call(**kw) == uns, kw
        for kw in (dict(q=P(A[0].value + 8)), dict(out=P(A[6].value + 4)), dict(ws=P(A[7].value + 8)), dict(stride=516),
                   dict(lens=P(A[4].value + 2)), dict(k=P(A[1].value + 8))):
            assert call(**kw) == mis, kw
        assert call(batch=0) == call(total=0, q=P(0)) == call(max_q=0) == Q.Q8A_OK
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1)):
        assert window(**kw) == bad, kw
    long = dict(max_kv=16 * 5000, width=5000, max_q=20, total=60, batch=3)
    assert window(window=30000, floats=10, **long) == bad and window(window=30000, ws=P(0), **long) == bad
    assert window(window=30000, ws=P(A[0].value + 64), **long) == bad and "overlap" in lib.q8a_last_error().decode()
    for kw in (dict(most=-1), dict(entries=-1), dict(entries=1 << 31), dict(most=161), dict(ptab=P(0)), dict(plen=P(0))):
        assert prefix(**kw) == bad, kw
    assert prefix(ptab=P(A[8].value + 1)) == mis and prefix(plen=P(A[9].value + 2)) == mis
    wide = dict(max_kv=16 * 50000, width=50000, entries=50000, most=16 * 40000, total=64, batch=64)
    assert prefix(floats=10, **wide) == bad and prefix(ws=P(0), **wide) == bad
    assert prefix(ws=P(A[6].value), **wide) == bad and "overlap" in lib.q8a_last_error().decode()
    for sizes in ((-1, 1, 8, 2, 1, 300), (1, 1, 7, 2, 1, 300), (1, 1, 8, 2, -1, 300)):
        assert lib.q8a_paged_window_workspace_floats(*sizes, 10, 0, 64) == -1
        assert lib.q8a_paged_prefix_workspace_floats(*sizes, 10, 64) == -1
    assert lib.q8a_paged_window_workspace_floats(1, 1, 8, 2, 1, 300, 0, 0, 64) == -1
    assert lib.q8a_paged_prefix_workspace_floats(1, 1, 8, 2, 1, 300, -1, 64) == -1
    assert lib.q8a_paged_window_workspace_floats(0, 1, 8, 2, 1, 300, 5, 0, 64) == 0
