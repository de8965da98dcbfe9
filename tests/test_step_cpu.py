"""Serving-step checks that need no GPU: symbols, struct layout, refusals, the oracle.

Validation happens on the host before any HIP call; device pointers here are fake addresses
that are never dereferenced.
"""
import ctypes
import os
import re
import subprocess
import sys
import tempfile

import numpy as np
import pytest

from oracle import step_oracle as so
from position_free_kv_amd import abi, step

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kamera_step.h")
FAKE = 0x10_0000_0000


def _gpu_present() -> bool:
    try:
        import torch
        return torch.cuda.device_count() > 0
    except Exception:  # noqa: BLE001
        return False


pytestmark = pytest.mark.skipif(_gpu_present(), reason="host-validation tests use fake device addresses")


def test_library_exports_every_declared_symbol():
    src = open(HEADER).read()
    names = set(re.findall(r"^(?:size_t|kamera_status) (kamera_\w+)\(", src, re.M))
    assert names == set(step.EXPORTED)
    for n in names:
        assert hasattr(abi.lib(), n), n


@pytest.mark.parametrize("lang,std", [("c", "c11"), ("c++", "c++11")])
def test_header_compiles_on_its_own(lang, std):
    cc = "gcc" if lang == "c" else "g++"
    r = subprocess.run([cc, f"-std={std}", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-x", lang, HEADER],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_structs_match_the_header():
    """Sizes and offsets of the binding's structs against the compiler's."""
    pairs = [("kamera_prefix", step.Prefix), ("kamera_request", step.Request), ("kamera_step", step.StepDesc),
             ("kamera_step_plan", step.Plan), ("kamera_append_rows", step.AppendRows)]
    body = "".join(f'printf("%zu ", sizeof({c}));' + "".join(f'printf("%zu ", offsetof({c}, {f}));' for f, _ in t._fields_)
                   for c, t in pairs)
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "a.c"), os.path.join(d, "a")
        open(src, "w").write(f'#include <stdio.h>\n#include "kamera_step.h"\nint main(void) {{{body} return 0;}}\n')
        subprocess.run(["gcc", "-I", os.path.dirname(HEADER), src, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = [x for _, t in pairs for x in [ctypes.sizeof(t)] + [getattr(t, f).offset for f, _ in t._fields_]]
    assert got == want
    assert step._REQUEST.itemsize == ctypes.sizeof(step.Request) and step._PREFIX.itemsize == ctypes.sizeof(step.Prefix)
    src = open(HEADER).read()
    for name, value in (("KAMERA_STEP_APPEND", step.APPEND), ("KAMERA_STEP_ATTEND", step.ATTEND), ("KAMERA_REQUEST_ALL", step.REQUEST_ALL),
                        ("KAMERA_ATTEND_MAX_DIM", step.ATTEND_MAX_DIM)):
        assert re.search(rf"{name} = {value}u?\b", src), name


# ------------------------------------------------------------------ refusals
GQA_LAY = dict(num_layers=2, num_kv_heads=2, head_dim=64, page_size=16)


def layout(**kw):
    return abi.make_layout(abi.GQA, abi.BF16, kw.pop("num_layers", 2), **{**{k: v for k, v in GQA_LAY.items() if k != "num_layers"}, **kw})


def pool(**kw):
    return abi.make_pool(kw.get("k", FAKE), kw.get("v", FAKE), kw.get("num_pages", 100), kw.get("layer_stride", 0))


def make(tables=((1, 2, 3),), num_tokens=40, num_queries=1, heads=4, **kw):
    return step.Step(num_q_heads=heads, block_tables=[np.array(t, np.int32) if t is not None else None for t in tables], num_tokens=num_tokens,
                     num_queries=num_queries, **kw)


def refused(name, fn, *args, **kw):
    with pytest.raises(abi.KameraError) as e:
        fn(*args, **kw)
    assert e.value.name == name and str(e.value) != f"{name}: ", str(e.value)


def upload(s, lay=None, p=None, ws=(FAKE, 1 << 30)):
    return step.upload(lay or layout(), s, p or pool(), ws)


PRE = [dict(block_table=np.array([7, 8], np.int32), num_tokens=20)]


@pytest.mark.parametrize("name,kw", [
    ("KAMERA_E_UNSUPPORTED", dict(flags=0)), ("KAMERA_E_UNSUPPORTED", dict(flags=8)),
    ("KAMERA_E_SHAPE", dict(heads=3)), ("KAMERA_E_SHAPE", dict(heads=0)), ("KAMERA_E_SHAPE", dict(heads=-2)),
    ("KAMERA_E_SHAPE", dict(num_tokens=-1)), ("KAMERA_E_SHAPE", dict(num_queries=-1)), ("KAMERA_E_SHAPE", dict(num_queries=41)),
    ("KAMERA_E_SHAPE", dict(prefix=0)), ("KAMERA_E_SHAPE", dict(prefix=-2)), ("KAMERA_E_PAGE", dict(slot0=16)), ("KAMERA_E_PAGE", dict(slot0=-1)),
    ("KAMERA_E_PAGE", dict(tables=((1, 2, 100),))), ("KAMERA_E_PAGE", dict(tables=((-1, 2, 3),))),
    ("KAMERA_E_UNSUPPORTED", dict(request_flags=2)),
    ("KAMERA_E_DELTA", dict(position0=(1 << 31) - 39)), ("KAMERA_E_DELTA", dict(position0=-(1 << 31))),
    ("KAMERA_E_PAGE", dict(prefix=0, prefixes=[dict(block_table=np.array([7, 100], np.int32), num_tokens=20)])),
    ("KAMERA_E_PAGE", dict(prefix=0, prefixes=[dict(block_table=np.array([7, 8], np.int32), num_tokens=20, slot0=16)])),
    ("KAMERA_E_SHAPE", dict(prefix=0, prefixes=[dict(block_table=np.array([7, 8], np.int32), num_tokens=-1)])),
    ("KAMERA_E_OVERLAP", dict(tables=((1, 2, 3), (4, 5, 3)))),  # both append to slot 7 of page 3
    ("KAMERA_E_OVERLAP", dict(tables=((1, 2, 2),), num_queries=30)),  # a page twice in one table
    ("KAMERA_E_OVERLAP", dict(tables=((1, 2, 8),), prefix=0, prefixes=[dict(block_table=np.array([7, 8], np.int32), num_tokens=24)])),
    ("KAMERA_E_ALIGN", dict(positions=FAKE + 2)),
])
def test_steps_refused(name, kw):
    refused(name, upload, make(**kw))


def test_null_pointers_pools_and_workspaces_refused():
    s = make()
    s.requests["block_table"] = 0
    refused("KAMERA_E_NULL", upload, s)
    s = make(prefix=0, prefixes=PRE)
    s.prefixes["block_table"] = 0
    refused("KAMERA_E_NULL", upload, s)
    refused("KAMERA_E_SHAPE", upload, make(num_tokens=(1 << 31) - 4000, num_queries=0))
    s = make()
    s.requests["reserved"] = 1
    refused("KAMERA_E_SHAPE", upload, s)
    for name, p in (("KAMERA_E_NULL", pool(k=None)), ("KAMERA_E_NULL", pool(v=None)), ("KAMERA_E_SHAPE", pool(num_pages=0)),
                    ("KAMERA_E_ALIGN", pool(k=FAKE + 1)), ("KAMERA_E_SHAPE", pool(layer_stride=100))):
        refused(name, upload, make(), p=p)
    f32 = abi.make_layout(abi.GQA, abi.F32, **GQA_LAY)  # (a bf16 layout's size covers two kernels)
    need = step.workspace_bytes(f32, make())
    assert need > 0
    refused("KAMERA_E_WORKSPACE", upload, make(), lay=f32, ws=(FAKE, need - 1))
    refused("KAMERA_E_WORKSPACE", upload, make(), ws=(FAKE, 256))
    refused("KAMERA_E_WORKSPACE", upload, make(), ws=None)
    refused("KAMERA_E_ALIGN", upload, make(), ws=(FAKE + 64, need))
    refused("KAMERA_E_SHAPE", upload, make(), lay=layout(head_dim=7))
    refused("KAMERA_E_UNSUPPORTED", upload, make(flags=step.ATTEND),
            lay=abi.make_layout(abi.MLA, abi.BF16, 1, latent_dim=1024, rope_dim=64))
    assert step.workspace_bytes(layout(), make(flags=0)) == 0
    assert step.workspace_bytes(layout(), make(num_tokens=-1)) == 0
    L = step._lib()
    assert L.kamera_step_workspace_bytes(None, None) == 0
    assert abi.STATUS[L.kamera_step_upload(None, None, None, None, 0, None, None)] == "KAMERA_E_NULL"
    assert abi.STATUS[L.kamera_step_append(None, 0, None, None)] == "KAMERA_E_NULL"
    assert abi.STATUS[L.kamera_step_attend(None, 0, None, 0, None, 0, None, 1.0, None)] == "KAMERA_E_NULL"


def test_appended_slots_may_share_a_page():
    """Two requests appending to different slots of one page, and one ending where a prefix page begins, are fine
    on the host (the upload then needs a GPU)."""
    s = make(tables=((1, 2, 3), (4, 5, 3)), num_tokens=[33, 40], num_queries=[1, 1])
    with pytest.raises(abi.KameraError) as e:
        upload(s)
    assert e.value.name == "KAMERA_E_HIP"
    s = make(tables=((1, 2, 8),), prefix=0, prefixes=PRE)  # prefix: slots 0-3 of page 8; appended: slot 7
    with pytest.raises(abi.KameraError) as e:
        upload(s)
    assert e.value.name == "KAMERA_E_HIP"


def empty_plan(flags=step.APPEND | step.ATTEND, family=abi.GQA):
    lay = layout() if family == abi.GQA else abi.make_layout(abi.MLA, abi.BF16, 2, latent_dim=64, rope_dim=16)
    plan = upload(make(num_queries=0, flags=flags), lay=lay)  # no tokens: nothing is enqueued
    plan.num_tokens = 1  # so that the launches' own checks are reached
    return plan


@pytest.mark.parametrize("name,kw", [
    ("KAMERA_E_NULL", dict(k=None)), ("KAMERA_E_NULL", dict(v=None)), ("KAMERA_E_NULL", dict(q=None)), ("KAMERA_E_NULL", dict(q_out=None)),
    ("KAMERA_E_ALIGN", dict(k=FAKE + 1)), ("KAMERA_E_ALIGN", dict(q=FAKE + 1)), ("KAMERA_E_ALIGN", dict(k_weight=FAKE + 1)),
    ("KAMERA_E_SHAPE", dict(k_stride=127)), ("KAMERA_E_SHAPE", dict(q_stride=255)), ("KAMERA_E_SHAPE", dict(v_stride=-1)),
    ("KAMERA_E_SHAPE", dict(q_out_stride=8)), ("KAMERA_E_SHAPE", dict(q_out=FAKE, q_out_stride=300)), ("KAMERA_E_SHAPE", dict(eps=-1.0)),
    ("KAMERA_E_SHAPE", dict(eps=float("nan"))), ("KAMERA_E_SHAPE", dict(layer=2)), ("KAMERA_E_SHAPE", dict(layer=-1))])
def test_append_refused(name, kw):
    args = dict(q=FAKE, q_out=FAKE + 4096, k=FAKE, v=FAKE, q_stride=0, k_stride=0, v_stride=0, q_out_stride=0)
    args.update(kw)
    refused(name, step.append, empty_plan(), args.pop("layer", 0), **args)


def test_append_refused_for_latent_rows_and_other_plans():
    args = dict(q=FAKE, q_out=FAKE, k=FAKE)
    refused("KAMERA_E_UNSUPPORTED", step.append, empty_plan(family=abi.MLA), 0, q_weight=FAKE, **args)
    refused("KAMERA_E_UNSUPPORTED", step.append, empty_plan(step.ATTEND), 0, v=FAKE, **args)
    refused("KAMERA_E_UNSUPPORTED", step.attend, empty_plan(step.APPEND), 0, FAKE, FAKE, 1.0)
    refused("KAMERA_E_WORKSPACE", step.append, step.Plan(), 0, v=FAKE, **args)


@pytest.mark.parametrize("name,kw", [
    ("KAMERA_E_NULL", dict(q=None)), ("KAMERA_E_NULL", dict(out=None)), ("KAMERA_E_ALIGN", dict(q=FAKE + 1)), ("KAMERA_E_ALIGN", dict(out=FAKE + 1)),
    ("KAMERA_E_ALIGN", dict(lse=FAKE + 2)), ("KAMERA_E_SHAPE", dict(q_stride=10)), ("KAMERA_E_SHAPE", dict(out_stride=255)),
    ("KAMERA_E_SHAPE", dict(scale=float("inf"))), ("KAMERA_E_SHAPE", dict(scale=float("nan"))), ("KAMERA_E_SHAPE", dict(layer=5))])
def test_attend_refused(name, kw):
    args = dict(layer=0, q=FAKE, out=FAKE, scale=1.0)
    args.update(kw)
    refused(name, step.attend, empty_plan(), args.pop("layer"), args.pop("q"), args.pop("out"), args.pop("scale"), **args)


def test_steps_without_tokens_do_nothing():
    plan = upload(make(tables=(), num_tokens=0, num_queries=0))
    assert plan.num_tokens == 0
    step.append(plan, 0, k=None)
    step.attend(plan, 1, None, None, 1.0)
    upload(make(tables=(None,), num_tokens=0, num_queries=0))


WS = (FAKE, 1 << 20)


def test_page_copies_refused():
    lay, p = layout(), pool()
    refused("KAMERA_E_PAGE", step.copy_pages, lay, p, [1], [100], WS)
    refused("KAMERA_E_PAGE", step.copy_pages, lay, p, [-1], [1], WS)
    refused("KAMERA_E_OVERLAP", step.copy_pages, lay, p, [1, 2], [3, 3], WS)
    refused("KAMERA_E_WORKSPACE", step.copy_pages, lay, p, [1, 2], [3, 4], (FAKE, step.copy_pages_workspace_bytes(2) - 1))
    refused("KAMERA_E_WORKSPACE", step.copy_pages, lay, p, [1], [3], None)
    refused("KAMERA_E_ALIGN", step.copy_pages, lay, p, [1], [3], (FAKE + 8, 1 << 20))
    refused("KAMERA_E_NULL", step.copy_pages, lay, pool(v=None), [1], [3], WS)
    with pytest.raises(ValueError):
        step.copy_pages(lay, p, [1, 2], [3], WS)
    L = step._lib()
    lb, pb = ctypes.byref(lay), ctypes.byref(p)
    assert abi.STATUS[L.kamera_copy_pages(lb, pb, None, None, 1, FAKE, 1 << 20, None)] == "KAMERA_E_NULL"
    assert abi.STATUS[L.kamera_copy_pages(lb, pb, None, None, -1, FAKE, 1 << 20, None)] == "KAMERA_E_SHAPE"
    assert L.kamera_copy_pages_workspace_bytes(-1) == 0
    step.copy_pages(lay, p, [], [], WS)
    step.copy_pages(lay, p, [4, 5], [4, 5], WS)  # nothing to do


def test_compaction_on_the_host():
    lay, p = layout(), pool()
    t = np.array([0, 2, 1, 1], np.int32)  # already together: no copy, tables as they were
    u = t.copy()
    assert step.compact_pages(lay, p, [u], WS) == 3 and np.array_equal(t, u)
    assert step.compact_pages(lay, p, [], WS) == 0
    refused("KAMERA_E_PAGE", step.compact_pages, lay, p, [np.array([100], np.int32)], WS)
    refused("KAMERA_E_WORKSPACE", step.compact_pages, lay, p, [np.array([5], np.int32)], (FAKE, 16))
    t = np.array([50, 1], np.int32)
    refused("KAMERA_E_HIP", step.compact_pages, lay, p, [t], WS)  # no GPU here: the tables stay
    assert t.tolist() == [50, 1]
    with pytest.raises(ValueError):
        step.compact_pages(lay, p, [np.array([1], np.int64)], WS)
    L = step._lib()
    lb, pb = ctypes.byref(lay), ctypes.byref(p)
    assert abi.STATUS[L.kamera_compact_pages(lb, pb, None, None, 1, None, FAKE, 1 << 20, None)] == "KAMERA_E_NULL"


@pytest.mark.parametrize("tables", [(np.zeros((3, 2), np.int32), 2), ([np.zeros(2, np.int32)], 2)])
def test_tables_and_requests_counted_alike(tables):
    with pytest.raises(ValueError):
        step._tables(*tables)


# ------------------------------------------------------------------ the oracle, against closed forms
def test_oracle_attention_is_a_mean_of_values_for_equal_scores():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((9, 4)), rng.standard_normal((9, 3))
    out, lse, absv, _ = so.attend(np.zeros((3, 2, 4)), k, v, 1.0, [8, 2, -1])
    assert np.allclose(out[0], v.mean(0)) and np.allclose(out[1], v[:3].mean(0)) and (out[2] == 0).all()
    assert np.allclose(lse[0], np.log(9)) and np.isneginf(lse[2]).all() and np.allclose(absv[0], np.abs(v).mean(0))
    q = rng.standard_normal((1, 1, 4))  # joined from two halves by their lse
    whole, z, _, _ = so.attend(q, k, v, 0.7, [8])
    (a, za, _, _), (b, zb, _, _) = so.attend(q, k[:4], v[:4], 0.7, [3]), so.attend(q, k[4:], v[4:], 0.7, [4])
    assert np.allclose(z, np.logaddexp(za, zb)) and np.allclose(whole, a * np.exp(za - z)[..., None] + b * np.exp(zb - z)[..., None])


def test_oracle_rotation_is_a_complex_product_and_norms_have_unit_mean_square():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 2, 8))
    phi = so.phases(np.arange(5) * 1000, 8, 1e4)
    y, t = so.rotate(x, phi)
    z = (x[..., :4] + 1j * x[..., 4:]) * np.exp(1j * phi)[:, None]
    assert np.allclose(y, np.concatenate([z.real, z.imag], -1)) and (t >= np.abs(y) - 1e-12).all()
    y, _ = so.rotate(x, phi, gptj=True)
    z = (x[..., ::2] + 1j * x[..., 1::2]) * np.exp(1j * phi)[:, None]
    assert np.allclose(y[..., ::2], z.real) and np.allclose(y[..., 1::2], z.imag)
    three = so.phases(np.array([[3, 50, 700]]), 8, 1e4, (1, 2, 1))
    assert np.allclose(three[0], np.array([3, 50, 50, 700]) * 1e4 ** (-np.arange(4) / 4))
    assert np.allclose((so.norm(x, np.ones(8), 0.0) ** 2).mean(-1), 1)


def test_work_lists_and_copy_orders():
    """tests/c_abi/step_host_check.cpp: the host part with stand-ins for the kernels, random steps and copy lists."""
    if os.environ.get("KAMERA_LIBRARY"):
        pytest.skip("no use of the loaded library")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "check")
        subprocess.run(["g++", "-std=c++17", "-O2", "-g", "-fsanitize=address", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include",
                        f"-I{os.path.join(ROOT, 'include')}", f"-I{os.path.join(ROOT, 'position_free_kv_amd', 'csrc')}",
                        os.path.join(ROOT, "tests", "c_abi", "step_host_check.cpp"),
                        os.path.join(ROOT, "position_free_kv_amd", "csrc", "kamera_step_host.cpp"), f"-L{rocm}/lib", "-lamdhip64",
                        f"-Wl,-rpath,{rocm}/lib", "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
        assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-2000:] + r.stderr[-2000:]


def test_host_code_under_address_sanitizer():
    """The refusals above against a build of the host parts with AddressSanitizer (device code is not instrumented)."""
    pkg = os.path.join(ROOT, "position_free_kv_amd")
    csrc, objs, rocm = os.path.join(pkg, "csrc"), os.path.join(pkg, "_build"), os.environ.get("ROCM_PATH", "/opt/rocm")
    if os.environ.get("KAMERA_LIBRARY"):
        pytest.skip("already inside")
    from position_free_kv_amd.build import STEP_KERNELS
    kernels = [os.path.join(objs, f + ".o") for f in ["kamera_kernels", "kamera_builder", "kamera_probe", *STEP_KERNELS]]
    libasan = subprocess.run(["gcc", "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    with tempfile.TemporaryDirectory() as d:
        hosts = []
        for name in ("kamera_host", "kamera_step_host"):
            hosts.append(os.path.join(d, name + ".o"))
            subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-fsanitize=address", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
                            f"-I{rocm}/include", f"-I{os.path.join(ROOT, 'include')}", f"-I{csrc}", "-c",
                            os.path.join(csrc, name + ".cpp"), "-o", hosts[-1]], check=True)
        lib = os.path.join(d, "libkamera_asan.so")
        subprocess.run(["g++", "-shared", "-fPIC", *kernels, *hosts, "-fsanitize=address", f"-L{rocm}/lib", "-lamdhip64",
                        f"-Wl,-rpath,{rocm}/lib", "-o", lib], check=True)
        env = dict(os.environ, LD_PRELOAD=libasan, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", KAMERA_LIBRARY=lib, PYTHONPATH=ROOT)
        r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", os.path.abspath(__file__)], env=env, cwd=ROOT,
                           capture_output=True, text=True, timeout=600)
        out = r.stdout + r.stderr
        assert r.returncode == 0 and "AddressSanitizer" not in out and " passed" in out, out[-3000:]
