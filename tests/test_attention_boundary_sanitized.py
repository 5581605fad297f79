"""The linear-attention boundary tests against the library whose host code runs under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only)."""

import glob
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="hipcc is needed to build the sanitized library")
def test_attention_boundary_runs_clean_under_asan_and_ubsan(tmp_path):
    from scan_primitives_amd import build_lib
    env = dict(os.environ)
    env.update({
        "SX_SCAN_LIB": build_lib.build_asan(),
        "LD_PRELOAD": build_lib.asan_runtime(),
        "ASAN_OPTIONS": f"detect_leaks=0:halt_on_error=1:log_path={tmp_path}/asan",
        "UBSAN_OPTIONS": f"halt_on_error=1:print_stacktrace=1:log_path={tmp_path}/ubsan",
    })
    proc = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_attention_boundary.py"),
                           "-q", "-p", "no:cacheprovider", "-m", "not gpu"], cwd=ROOT, env=env, capture_output=True,
                          text=True, timeout=600)
    reports = sorted(glob.glob(str(tmp_path / "asan*")) + glob.glob(str(tmp_path / "ubsan*")))
    assert not reports, "".join(open(r).read() for r in reports)[:4000]
    assert proc.returncode == 0, proc.stdout[-3000:] + proc.stderr[-3000:]
    assert " passed" in proc.stdout
