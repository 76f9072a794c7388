"""The host code of the step's calls and of the window's and the prefix's attention under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_paged_abi_sanitized.py does for the other paged calls.  CPU only."""

import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT
from tests.test_abi_sanitized import _runtime


def test_step_and_range_abi_under_asan_and_ubsan():
    asan = _runtime("libasan.so")
    if asan is None:
        pytest.skip("no AddressSanitizer runtime for this compiler")
    from chunked_prefill_attention_gb300 import _build
    _build.ensure_built()   # the sanitized library shares its kernels' objects
    env = dict(os.environ, LD_PRELOAD=asan, Q8ATTN_LIBRARY=_build.build_sanitized(),
               ASAN_OPTIONS="protect_shadow_gap=0:detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    tests = [os.path.join(ROOT, "tests", f) for f in ("test_paged_step_abi_cpu.py", "test_paged_range_cpu.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", *tests], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    out = r.stdout[-3000:] + r.stderr[-3000:]
    assert r.returncode == 0, out
    assert "AddressSanitizer" not in out and "runtime error" not in out, out
    assert " passed" in r.stdout and "skipped" not in r.stdout, out
