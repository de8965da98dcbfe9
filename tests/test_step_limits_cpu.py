"""Limits of the serving step's host part, on the CPU."""
import os
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_part_at_its_limits():
    """tests/c_abi/step_limits_check.cpp under AddressSanitizer (no device code in it)."""
    if os.environ.get("KAMERA_LIBRARY"):
        pytest.skip("no use of the loaded library")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    csrc = os.path.join(ROOT, "position_free_kv_amd", "csrc")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "check")
        subprocess.run(["g++", "-std=c++17", "-O2", "-g", "-fsanitize=address", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include",
                        f"-I{os.path.join(ROOT, 'include')}", f"-I{csrc}", os.path.join(ROOT, "tests", "c_abi", "step_limits_check.cpp"),
                        os.path.join(csrc, "kamera_step_host.cpp"), f"-L{rocm}/lib", "-lamdhip64", f"-Wl,-rpath,{rocm}/lib", "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
        assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-2000:] + r.stderr[-2000:]
