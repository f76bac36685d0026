"""tests/host/gr_plan_bounds.cpp, the bounds harness of the plans in ss_gr_plan.h, under AddressSanitizer and
UndefinedBehaviorSanitizer (every finding fatal).  Its self-test must report a planted overlap.  No GPU is
involved."""
import shutil
import subprocess

import pytest

from tests.test_sanitize import ENV, ROOT, SAN, _build


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_gr_plan_bounds_sanitized(tmp_path):
    exe = str(tmp_path / "gr_plan_bounds")
    _build(["g++", "-std=c++17", *SAN, f"-I{ROOT}/include", f"-I{ROOT}/selective_state_space_34_amd/csrc",
            "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", f"{ROOT}/tests/host/gr_plan_bounds.cpp", "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=ENV)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.startswith("gr plan bounds ok") and int(r.stdout.split()[-1]) > 200000, r.stdout
    planted = subprocess.run([exe, "selftest"], capture_output=True, text=True, timeout=60, env=ENV)
    assert planted.returncode == 1 and "FAIL" in planted.stdout, planted.stdout
