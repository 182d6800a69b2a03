"""The serving entry points' host-side argument validation (sizes, strides, the
struct of scored rows) under AddressSanitizer and UndefinedBehaviorSanitizer:
their host tests against a library built with the host sanitizers, in a child
process that preloads the compiler's runtime (CPU only, no kernel is launched)."""
import os
import subprocess
import sys

import pytest

from invariant_token_log_fp32_amd import build

pytestmark = pytest.mark.slow


def test_serving_validation_is_clean_under_asan_and_ubsan(tmp_path):
    runtime = build.asan_runtime()
    if not runtime:
        pytest.skip("the compiler's AddressSanitizer runtime was not found")
    lib = build.build_host_sanitized(str(tmp_path / "librlk_logp.so"))
    env = dict(os.environ, RLK_LIBRARY=lib, LD_PRELOAD=runtime,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "tests/test_mx4_host.py",
                          "tests/test_draft_host.py", "tests/test_serving_sizes_host.py"],
                         cwd=root, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert " passed" in out
