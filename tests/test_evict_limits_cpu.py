"""Limits of eviction, weighing and differential attention, on the CPU: what a launch shares out, what is refused."""
import os
import subprocess
import tempfile

import numpy as np
import pytest

from position_free_kv_amd import abi, step

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "position_free_kv_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
FAKE = 0x10_0000_0000


def _gpu_present() -> bool:
    try:
        import torch
        return torch.cuda.device_count() > 0
    except Exception:  # noqa: BLE001
        return False


pytestmark = pytest.mark.skipif(_gpu_present(), reason="fake device addresses")


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


@pytest.mark.parametrize("family,layers,seqs,keep,flags,fits", [
    (abi.MLA, 1 << 20, 2047, 0, 0, True), (abi.MLA, 1 << 20, 2048, 0, 0, False),                    # lists
    (abi.GQA, 1 << 15, 1023, 1, 0, True), (abi.GQA, 1 << 15, 1024, 1, 0, False),                    # 64 workgroups each that move rows
    (abi.MLA, 1 << 18, 910, 1, step.REANCHOR, True), (abi.MLA, 1 << 18, 911, 1, step.REANCHOR, False)])  # 9 each
def test_evictions_of_more_than_one_launch_are_refused(family, layers, seqs, keep, flags, fits):
    """Before anything is enqueued: scores that have moved without their rows could not be put right."""
    kind = dict(num_kv_heads=8, head_dim=256) if family == abi.GQA else dict(latent_dim=512, rope_dim=64)
    lay = abi.make_layout(family, abi.BF16, layers, page_size=2, **kind)
    e = step.Eviction(block_tables=np.arange(seqs, dtype=np.int32).reshape(seqs, 1), num_tokens=2, keep=keep, flags=flags)
    with pytest.raises(abi.KameraError) as err:
        step.evict(lay, abi.make_pool(FAKE, FAKE if family == abi.GQA else None, seqs), e, FAKE, (FAKE, 1 << 50))
    assert err.value.name == ("KAMERA_E_HIP" if fits else "KAMERA_E_SHAPE")


def test_long_requests_among_short_ones_are_shared_out():
    compiled_and_run("diff_plan_check.cpp", "kamera_step_host.cpp", "kamera_evict_host.cpp")


@pytest.mark.parametrize("flags", [0, step.REANCHOR])
@pytest.mark.parametrize("family,page", [(abi.GQA, 1), (abi.GQA, 16), (abi.MLA, 3), (abi.MLA, 64)])
def test_a_workspace_serves_shorter_evictions(family, page, flags):
    """Of some of the sequences, each of at most as many tokens that keeps at most as many, wherever they begin in a page."""
    kind = dict(num_kv_heads=2, head_dim=128) if family == abi.GQA else dict(latent_dim=512, rope_dim=64)
    lay = abi.make_layout(family, abi.BF16, 2, page_size=page, **kind)
    rng = np.random.default_rng(page)

    def eviction(n, keep):
        slot0 = rng.integers(0, page, n.size)
        entries = -(-(slot0 + n) // page)
        tables = np.split(np.arange(entries.sum(), dtype=np.int32), np.cumsum(entries)[:-1])
        return step.Eviction(block_tables=tables, num_tokens=n, keep=keep, slot0=slot0, flags=flags)

    pool = abi.make_pool(FAKE, FAKE if family == abi.GQA else None, 1 << 20)
    cases = [([1100], [1090], [1000], [100]), ([2000], [2000], [1000], [100]), ([8000], [7900], [4000], [500]), ([1600], [1600], [1599], [1599])]
    for _ in range(60):
        seqs = int(rng.integers(1, 12))
        n = np.exp(rng.uniform(0, np.log(9000), seqs)).astype(np.int64)
        keep = np.exp(rng.uniform(0, np.log(9000), seqs)).astype(np.int64)
        some = rng.random(seqs) < 0.7
        some[rng.integers(seqs)] = True
        cases.append((n, keep, rng.integers(1, n[some] + 1), rng.integers(0, keep[some] + 1)))
    for n, keep, less, stay in cases:
        large, small = eviction(np.asarray(n), keep), eviction(np.asarray(less), stay)
        room = step.evict_workspace_bytes(lay, large)
        assert 0 < step.evict_workspace_bytes(lay, small) <= room, (n, keep, less, stay)
        try:
            step.evict(lay, pool, small, FAKE, (FAKE, room))
        except abi.KameraError as e:  # (staging needs a GPU)
            assert e.name == "KAMERA_E_HIP", e


def test_rows_are_left_whole_in_small_workspaces():
    compiled_and_run("weigh_plan_check.cpp", "kamera_step_host.cpp", "kamera_evict_host.cpp")
