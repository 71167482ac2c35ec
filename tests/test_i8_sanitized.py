"""tests/test_i8_checks.py re-run against a build whose host code carries AddressSanitizer and
UndefinedBehaviorSanitizer checks, as tests/test_sanitizers.py does with the other CPU tests of the C ABI."""
from __future__ import annotations

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_i8_checks_pass_under_asan_and_ubsan():
    import sanitized_build as sb

    env = dict(os.environ)
    env.update({
        "LD_PRELOAD": sb.asan_runtime(),
        "ASAN_OPTIONS": "detect_leaks=0:abort_on_error=1:halt_on_error=1",
        "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1",
        "QUEST_LIBRARY": sb.build_sanitized(),
    })
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "not gpu", "-p", "no:cacheprovider",
                          os.path.join(ROOT, "tests", "test_i8_checks.py")],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = res.stdout + res.stderr
    assert "Sanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert res.returncode == 0, out[-4000:]
