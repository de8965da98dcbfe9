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


def test_flag_of_plans_that_fit_their_workspace():
    import re

    import numpy as np

    from position_free_kv_amd import abi, step
    assert re.search(rf"KAMERA_STEP_FIT = {step.FIT}u\b", open(os.path.join(ROOT, "include", "kamera_step.h")).read())
    lay = abi.make_layout(abi.GQA, abi.BF16, 1, num_kv_heads=8, head_dim=128, page_size=16)
    s = step.Step(num_q_heads=32, block_tables=[np.zeros(300, np.int32)], num_tokens=1, num_queries=1, flags=step.FIT)
    assert step.workspace_bytes(lay, s) == 0  # nothing to launch

    def size(requests, tokens, queries, flags):
        return step.workspace_bytes(lay, step.Step(num_q_heads=32, block_tables=np.zeros((requests, 300), np.int32), num_tokens=tokens, num_queries=queries,
                                                   prefix=0, prefixes=[dict(block_table=np.zeros(512, np.int32), num_tokens=8192)], flags=flags))
    for flags in (step.ATTEND, step.ATTEND | step.FIT):  # the sizes of the fastest plans fall as steps grow
        assert size(64, 64, 1, flags) > size(64, 4192, 1, flags) and size(8, 1000, 23, flags) > size(8, 1000, 256, flags)
