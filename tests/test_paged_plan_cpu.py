"""What attn_paged launches against the workspace it accepts (no GPU needed): the library runs in a child process
whose launches are replaced, so that every plan can be looked at and nothing reaches a device."""

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

    def run(cases):
        r = subprocess.run([sys.executable, "-c", "import sys, json; from tests.test_paged_plan_cpu import child; "
                                                  "child(json.load(sys.stdin))"],
                           cwd=ROOT, env=dict(os.environ, LD_PRELOAD=so), input=json.dumps(cases), capture_output=True,
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
