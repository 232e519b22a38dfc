"""The microscaled 4-bit and expert entry points' host code under
AddressSanitizer and UndefinedBehaviorSanitizer: their CPU refusal tests run
against liblutq_san.so with the clang ASan runtime preloaded. Any sanitizer
report fails the run."""

import os
import subprocess
import sys

import pytest

from weight_only_lut_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_refusals_clean_under_host_sanitizers():
    runtime = build.asan_runtime()
    if runtime is None:
        pytest.skip("clang ASan runtime not found")
    if not os.path.exists(build.SAN_LIB):
        pytest.skip("liblutq_san.so not built (python -m weight_only_lut_amd.build)")
    env = dict(os.environ)
    env.update({"LUTQ_LIBRARY": build.SAN_LIB, "LD_PRELOAD": runtime,
                "ASAN_OPTIONS": "detect_leaks=0:abort_on_error=1",
                "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"})
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                          os.path.join(ROOT, "tests", "test_abi_mx.py")],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-3000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-3000:]
    assert " passed" in out
