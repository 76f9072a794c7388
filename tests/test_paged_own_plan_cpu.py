"""How attn_paged_prefix cuts the keys behind the prefix (no GPU needed).  The prefix's length is the device's, anything from 0 to
its bound, so a sequence's own keys may be all that max_kv allows: the plan of a call that shares must not leave those to a few
blocks.  The launches run in a child process where they are replaced."""

import ctypes
import itertools
import json
import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT

P = ctypes.c_void_p
SMS = 152


def child(cases):
    """Runs in the child: how each call's own keys are cut."""
    from chunked_prefill_attention_gb300 import q8attn as Q
    lib, rec, out = Q.load(), ctypes.CDLL(None), []
    rec.record_own.argtypes = [P]
    got = (ctypes.c_int64 * 9)()
    rec.record_own(got)
    for batch, q, group, kv, D, max_kv, most, *rows in cases:
        page, heads = 64, kv * group
        total = rows[0] if rows else batch * q
        floats = lib.q8a_paged_prefix_workspace_floats(batch, total, heads, kv, q, max_kv, most, D)
        rc = lib.attn_paged_prefix(P(1 << 36), 0, heads * D, total, heads, kv, D, P(0x200000), P(0x300000), 4, page,
                                   kv * page * D // 32 * 34, P(0x400000), -(-max_kv // page), P(0x500000), P(0x600000), batch, q,
                                   max_kv, P(0x800000), -(-most // page), P(0x900000), most, 0.125, 1, P(1 << 38),
                                   P(0x7000000000), floats, P(0))
        assert rc == 0, lib.q8a_last_error()
        rec.record_own(got)
        out.append(dict(zip(("kind", "direct", "cluster", "row_tiles", "rows", "shares", "ctas", "shared", "only"), got)))
    print(json.dumps(out))


@pytest.fixture(scope="module")
def plans(lib, tmp_path_factory):
    so = str(tmp_path_factory.mktemp("record") / "record.so")
    cuda = next((p for p in ("/usr/local/cuda/include", os.path.join(os.environ.get("CUDA_HOME", ""), "include"))
                 if os.path.exists(os.path.join(p, "cuda_runtime.h"))), None)
    if cuda is None:
        pytest.skip("no CUDA headers")
    r = subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", cuda, "-I", os.path.join(ROOT, "include"), "-o", so,
                        os.path.join(ROOT, "tests", "paged_own_record.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases):
        r = subprocess.run([sys.executable, "-c", "import sys, json; from tests.test_paged_own_plan_cpu import child; "
                                                  "child(json.load(sys.stdin))"],
                           cwd=ROOT, env=dict(os.environ, LD_PRELOAD=" ".join([os.environ.get("LD_PRELOAD", ""), so]).strip()),
                           input=json.dumps(cases), capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        return json.loads(r.stdout)

    return run


def test_own_keys_are_planned_for_short_prefixes_too(plans):
    """Bounds that leave few own keys beside a long prefix: the clusters of few rows fill their wave or are as large as
    they get, and the tile kernel's units are cut where there are few of them."""
    cases = [(batch, q, 4, kv, D, most + own, most) for batch, q, kv, D, own, most in itertools.product(
        (3, 4, 8, 16, 30, 64, 200), (1, 4, 8, 16, 32), (1, 2, 8), (64, 128), (1, 200, 768, 2000), (32000, 400000))]
    few = tiles = 0
    for case, p in zip(cases, plans(cases)):
        batch, q, group, kv, D, max_kv, most = case
        if not p["shared"]:
            continue
        if p["kind"] == 0 and p["direct"]:
            few += 1
            ctas = batch * kv * p["row_tiles"] * p["cluster"]
            # the instance with an SM for each CTA, where the grid leaves one
            assert p["only"] == (p["rows"] > 8 and D == 128 and batch * kv * p["row_tiles"] <= SMS), (case, p)
            wave = SMS * (1 if p["only"] else 2)
            assert 2 * ctas > wave or p["cluster"] == (8 if p["rows"] <= 8 else 4), (case, p)
            assert p["cluster"] == 1 or ctas <= wave, (case, p)
        elif p["kind"] == 1 and batch <= 64:
            tiles += 1
            units = batch * kv * -(-q * group // 128)
            assert units > 2 * SMS // 3 or (p["shares"] and p["ctas"] >= SMS), (case, p)
    assert few > 100 and tiles > 50


def test_clusters_of_a_call_with_few_sequences(plans):
    for batch, q, kv, D, cluster in ((4, 1, 8, 128, 8), (8, 1, 8, 128, 4), (16, 1, 8, 128, 2), (64, 1, 8, 128, 1), (4, 4, 8, 128, 4),
                                     (16, 4, 8, 64, 2)):
        assert plans([(batch, q, 4, kv, D, 32768, 32000)])[0]["cluster"] == cluster, (batch, q, kv, D)


def test_which_batches_share(plans):
    """Of the batches that tests/test_gpu_paged_range.py calls behind a prefix of any length, those that share it: with bounds of
    2^19 keys all but one sequence, two single tokens, three of one K/V head of 64 channels, and rows that fill the tiles by
    themselves; with their own bounds only two large ones."""
    pytest.importorskip("torch")
    from tests.test_gpu_paged_range import PREFIX

    def shared(bounds):
        return [i for i, p in enumerate(plans([(len(q), max(q), heads // kv, kv, D, *bounds(prefix, max(own), page), sum(q))
                                               for q, own, prefix, heads, kv, D, page in PREFIX])) if p["shared"]]

    loose = shared(lambda prefix, own, page: ((1 << 19) + own, 1 << 19))
    assert [PREFIX[i][0] for i in range(len(PREFIX)) if i not in loose] == [[1, 1], [1, 1, 1], [200, 3], [7]]
    assert [PREFIX[i][0] for i in shared(lambda prefix, own, page: (prefix + own, -(-prefix // page) * page))] == [[1] * 300, [5] * 40]


def test_a_prefix_of_any_length_is_planned_for_any(plans):
    """max_prefix = max_kv: the own keys in shares, few rows or tiles, however many sequences fill the wave."""
    for batch, q, kv, D in ((64, 1, 8, 128), (16, 1, 8, 64), (16, 4, 8, 128), (16, 8, 8, 64), (16, 8, 8, 128), (4, 16, 8, 128)):
        p = plans([(batch, q, 4, kv, D, 32768, 32768)])[0]
        assert p["shared"] and (not p["direct"] if p["kind"] == 0 else p["shares"]), (batch, q, kv, D, p)
