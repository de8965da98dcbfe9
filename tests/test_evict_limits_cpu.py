"""Limits of eviction, weighing and differential attention, on the CPU: what a launch shares out, what is refused."""
import os
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "position_free_kv_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def compiled_and_run(check: str, *sources: str) -> None:
    """tests/c_abi/<check> under AddressSanitizer (no device code in it)."""
    if os.environ.get("KAMERA_LIBRARY"):
        pytest.skip("no use of the loaded library")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "check")
        subprocess.run(["g++", "-std=c++17", "-O2", "-g", "-fsanitize=address", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                        f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(ROOT, "tests", "c_abi", check),
                        *[os.path.join(CSRC, s) for s in sources], f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib", "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
        assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-2000:] + r.stderr[-2000:]


def test_every_workgroup_of_a_move_has_work_of_its_own_or_none():
    compiled_and_run("evict_moves_check.cpp")
