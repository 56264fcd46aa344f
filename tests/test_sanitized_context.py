"""The context operators' host code (argument checks, sizes) under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): their CPU tests in
a child process that loads the sanitizer build of the library."""
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
sys.path.insert(0, os.path.join(HERE, "sanitize"))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
@pytest.mark.skipif("PKV_LIBRARY" in os.environ, reason="already inside a sanitized run")
def test_context_host_code_under_asan_and_ubsan():
    import build_sanitized
    import build_sanitized_context

    lib = build_sanitized_context.build()
    asan = build_sanitized.asan_runtime()
    if not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("g++ has no ASan runtime")
    env = dict(os.environ, PKV_LIBRARY=lib, LD_PRELOAD=asan,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "tests/test_context_capi.py", "-q", "-s",
                          "-p", "no:cacheprovider"],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert res.returncode == 0 and " passed" in out and "skipped" not in out, out[-4000:]
