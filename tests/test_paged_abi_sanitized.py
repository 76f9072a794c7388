"""The host code of the paged calls (argument checks, plans, overlaps) under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_abi_sanitized.py does for the other calls.  CPU only."""

import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT
from tests.test_abi_sanitized import _runtime


def test_paged_abi_under_asan_and_ubsan():
    asan = _runtime("libasan.so")
    if asan is None:
        pytest.skip("no AddressSanitizer runtime for this compiler")
    from chunked_prefill_attention_gb300 import _build
    _build.ensure_built()   # the sanitized library shares its kernels' objects
    env = dict(os.environ, LD_PRELOAD=asan, Q8ATTN_LIBRARY=_build.build_sanitized(),
               ASAN_OPTIONS="protect_shadow_gap=0:detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    tests = [os.path.join(ROOT, "tests", f) for f in ("test_paged_abi_cpu.py", "test_paged_plan_cpu.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", *tests], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    out = r.stdout[-3000:] + r.stderr[-3000:]
    assert r.returncode == 0, out
    assert "AddressSanitizer" not in out and "runtime error" not in out, out
    assert " passed" in r.stdout and "skipped" not in r.stdout, out
