"""Differential attention, weighing and eviction without a GPU: struct layout, refusals, host parts, the oracle.

Validation happens on the host before any HIP call; device pointers here are fake addresses
that are never dereferenced.
"""
import os
import re
import subprocess
import tempfile

import numpy as np
import pytest

from oracle import evict_oracle as eo
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


def test_structs_and_constants_match_the_header():
    pairs = [("kamera_differential", step.Differential), ("kamera_evict_seq", step.EvictSeq), ("kamera_eviction", step.EvictDesc)]
    body = "".join(f'printf("%zu ", sizeof({c}));' + "".join(f'printf("%zu ", offsetof({c}, {f}));' for f, _ in t._fields_) for c, t in pairs)
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "a.c"), os.path.join(d, "a")
        open(src, "w").write(f'#include <stdio.h>\n#include "kamera_step.h"\nint main(void) {{{body} return 0;}}\n')
        subprocess.run(["gcc", "-I", os.path.dirname(HEADER), src, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    import ctypes
    want = []
    for _, t in pairs:
        want += [ctypes.sizeof(t)] + [getattr(t, f).offset for f, _ in t._fields_]
    assert got == want
    text = open(HEADER).read()
    for name, value in (("KAMERA_STEP_WEIGH", step.WEIGH), ("KAMERA_STEP_DIFFERENTIAL", step.DIFFERENTIAL), ("KAMERA_DIFF_NORM", step.DIFF_NORM),
                        ("KAMERA_EVICT_REANCHOR", step.REANCHOR)):
        assert re.search(rf"{name} = {value}u\b", text)


def test_host_parts():
    """tests/c_abi/evict_host_check.cpp under AddressSanitizer (no device code in it)."""
    if os.environ.get("KAMERA_LIBRARY"):
        pytest.skip("no use of the loaded library")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    csrc = os.path.join(ROOT, "position_free_kv_amd", "csrc")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "check")
        subprocess.run(["g++", "-std=c++17", "-O2", "-g", "-fsanitize=address", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include",
                        f"-I{os.path.join(ROOT, 'include')}", f"-I{csrc}", os.path.join(ROOT, "tests", "c_abi", "evict_host_check.cpp"),
                        os.path.join(csrc, "kamera_step_host.cpp"), os.path.join(csrc, "kamera_evict_host.cpp"), f"-L{rocm}/lib", "-lamdhip64",
                        f"-Wl,-rpath,{rocm}/lib", "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
        assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-2000:] + r.stderr[-2000:]


# ------------------------------------------------------------------ refusals
def refused(name, f, *a, **kw):
    with pytest.raises(abi.KameraError) as e:
        f(*a, **kw)
    assert e.value.name == name, e.value


def layout(family=abi.GQA, **kw):
    base = dict(num_kv_heads=4, head_dim=64) if family == abi.GQA else dict(latent_dim=64, rope_dim=16)
    return abi.make_layout(family, abi.BF16, 2, **{**base, "page_size": 16, **kw})


def a_step(flags, heads=8, **kw):
    return step.Step(num_q_heads=heads, block_tables=[np.array([1, 2, 3], np.int32)], num_tokens=40, num_queries=kw.pop("num_queries", 0), flags=flags, **kw)


def plan_of(flags, lay=None, **kw):
    lay = lay or layout()
    plan = step.upload(lay, a_step(flags, **kw), abi.make_pool(FAKE, FAKE, 100), (FAKE, 1 << 30))  # no tokens: nothing is enqueued
    plan.num_tokens = 1  # so that the launches' own checks are reached
    return plan


def test_steps_refused():
    up = lambda flags, lay, **kw: step.upload(lay, a_step(flags, **kw), abi.make_pool(FAKE, FAKE, 100), (FAKE, 1 << 30))  # noqa: E731
    both = step.ATTEND | step.DIFFERENTIAL
    refused("KAMERA_E_UNSUPPORTED", up, step.DIFFERENTIAL, layout())
    refused("KAMERA_E_UNSUPPORTED", up, step.APPEND | step.DIFFERENTIAL, layout())
    refused("KAMERA_E_UNSUPPORTED", up, step.ATTEND | 64, layout())
    refused("KAMERA_E_UNSUPPORTED", up, both, layout(num_kv_heads=1))
    refused("KAMERA_E_UNSUPPORTED", up, both, layout(abi.MLA))
    refused("KAMERA_E_SHAPE", up, both, layout(), heads=6)
    refused("KAMERA_E_SHAPE", up, step.WEIGH, layout(), heads=0)
    refused("KAMERA_E_SHAPE", up, step.WEIGH, layout(), heads=6)
    refused("KAMERA_E_UNSUPPORTED", up, step.WEIGH, layout(abi.MLA, latent_dim=1024))
    s = step.Step(num_q_heads=8, block_tables=[np.array([1, 2, 1], np.int32)], num_tokens=40, num_queries=1, flags=step.WEIGH)
    refused("KAMERA_E_OVERLAP", step.upload, layout(), s, abi.make_pool(FAKE, FAKE, 100), (FAKE, 1 << 30))
    assert step.workspace_bytes(layout(), a_step(both, num_queries=1)) > 0
    assert step.workspace_bytes(layout(abi.MLA), a_step(both, num_queries=1)) == 0


@pytest.mark.parametrize("name,kw", [
    ("KAMERA_E_NULL", dict(q=None)), ("KAMERA_E_NULL", dict(out=None)), ("KAMERA_E_ALIGN", dict(q=FAKE + 1)), ("KAMERA_E_ALIGN", dict(lse=FAKE + 2)),
    ("KAMERA_E_ALIGN", dict(lambdas=FAKE + 2)), ("KAMERA_E_ALIGN", dict(norm_weight=FAKE + 1)), ("KAMERA_E_SHAPE", dict(q_stride=511)),
    ("KAMERA_E_SHAPE", dict(out_stride=511)), ("KAMERA_E_SHAPE", dict(out_stride=-1)), ("KAMERA_E_SHAPE", dict(scale=float("inf"))),
    ("KAMERA_E_SHAPE", dict(lambda_init=float("nan"))), ("KAMERA_E_SHAPE", dict(out_scale=float("inf"))), ("KAMERA_E_SHAPE", dict(eps=-1.0)),
    ("KAMERA_E_SHAPE", dict(eps=float("nan"))), ("KAMERA_E_SHAPE", dict(layer=2)), ("KAMERA_E_SHAPE", dict(layer=-1))])
def test_attend_diff_refused(name, kw):
    kw = dict(dict(layer=0, q=FAKE, out=FAKE, scale=1.0, lambda_init=0.5), **kw)
    refused(name, step.attend_diff, plan_of(step.ATTEND | step.DIFFERENTIAL), kw.pop("layer"), kw.pop("q"), kw.pop("out"), kw.pop("scale"), **kw)


def test_launches_of_other_steps_refused():
    refused("KAMERA_E_UNSUPPORTED", step.attend_diff, plan_of(step.ATTEND), 0, FAKE, FAKE, 1.0, lambda_init=0.5)
    refused("KAMERA_E_UNSUPPORTED", step.attend_diff, plan_of(step.WEIGH | step.DIFFERENTIAL), 0, FAKE, FAKE, 1.0, lambda_init=0.5)
    refused("KAMERA_E_UNSUPPORTED", step.attend, plan_of(step.ATTEND | step.DIFFERENTIAL), 0, FAKE, FAKE, 1.0)
    refused("KAMERA_E_UNSUPPORTED", step.weigh, plan_of(step.ATTEND), 0, FAKE, FAKE, FAKE, 1.0)
    L = step._lib()
    assert abi.STATUS[L.kamera_step_attend_diff(None, 0, None, 0, None, 0, None, 1.0, None, None)] == "KAMERA_E_NULL"
    import ctypes
    assert abi.STATUS[L.kamera_step_attend_diff(ctypes.byref(plan_of(step.ATTEND | step.DIFFERENTIAL)), 0, FAKE, 0, FAKE, 0, None, 1.0, None, None)] == "KAMERA_E_NULL"
    d = step.Differential(None, None, 0.5, 0.5, 1e-5, 2)
    assert abi.STATUS[L.kamera_step_attend_diff(ctypes.byref(plan_of(step.ATTEND | step.DIFFERENTIAL)), 0, FAKE, 0, FAKE, 0, None, 1.0, ctypes.byref(d), None)] == "KAMERA_E_UNSUPPORTED"
    assert abi.STATUS[L.kamera_step_weigh(None, 0, None, 0, None, None, 1.0, 1.0, None)] == "KAMERA_E_NULL"
    assert abi.STATUS[L.kamera_evict(None, None, None, None, 0, None)] == "KAMERA_E_NULL"
    assert L.kamera_evict_workspace_bytes(None, None) == 0
    assert abi.STATUS[L.kamera_scores_layout(None, None)] == "KAMERA_E_NULL"
    assert abi.STATUS[L.kamera_scores_layout(ctypes.byref(layout()), None)] == "KAMERA_E_NULL"


@pytest.mark.parametrize("name,kw", [
    ("KAMERA_E_NULL", dict(q=None)), ("KAMERA_E_NULL", dict(lse=None)), ("KAMERA_E_NULL", dict(scores=None)), ("KAMERA_E_ALIGN", dict(q=FAKE + 1)),
    ("KAMERA_E_ALIGN", dict(lse=FAKE + 2)), ("KAMERA_E_ALIGN", dict(scores=FAKE + 1)), ("KAMERA_E_SHAPE", dict(q_stride=511)),
    ("KAMERA_E_SHAPE", dict(scale=float("nan"))), ("KAMERA_E_SHAPE", dict(decay=float("inf"))), ("KAMERA_E_SHAPE", dict(layer=2))])
def test_weigh_refused(name, kw):
    kw = dict(dict(layer=0, q=FAKE, lse=FAKE, scores=FAKE, scale=1.0), **kw)
    refused(name, step.weigh, plan_of(step.WEIGH), kw.pop("layer"), kw.pop("q"), kw.pop("lse"), kw.pop("scores"), kw.pop("scale"), **kw)


def eviction(tables=((1, 2, 3), (4, 5, 6)), **kw):
    args = dict(num_tokens=40, keep=20, first=2, last=3)
    args.update(kw)
    return step.Eviction(block_tables=[np.array(t, np.int32) for t in tables], **args)


def evict(e, lay=None, pool=None, scores=FAKE, ws=(FAKE, 1 << 30), **kw):
    step.evict(lay or layout(), pool or abi.make_pool(FAKE, FAKE, 100), e, scores, ws, **kw)


@pytest.mark.parametrize("name,kw", [
    ("KAMERA_E_SHAPE", dict(num_tokens=-1)), ("KAMERA_E_SHAPE", dict(keep=-1)), ("KAMERA_E_SHAPE", dict(first=-1)), ("KAMERA_E_SHAPE", dict(last=-1)),
    ("KAMERA_E_SHAPE", dict(first=18, last=3)), ("KAMERA_E_SHAPE", dict(first=2 ** 31 - 1, last=2 ** 31 - 1)), ("KAMERA_E_PAGE", dict(slot0=16)),
    ("KAMERA_E_PAGE", dict(slot0=-1)), ("KAMERA_E_PAGE", dict(tables=((1, 2, 100),))), ("KAMERA_E_PAGE", dict(tables=((-1, 2, 3),))),
    ("KAMERA_E_OVERLAP", dict(tables=((1, 2, 3), (4, 3, 5)))), ("KAMERA_E_OVERLAP", dict(tables=((1, 2, 1),))),
    ("KAMERA_E_SHAPE", dict(heads_together=0)), ("KAMERA_E_SHAPE", dict(heads_together=3)), ("KAMERA_E_UNSUPPORTED", dict(flags=2))])
def test_evictions_refused(name, kw):
    refused(name, evict, eviction(**kw))


def test_evictions_arguments_refused():
    e = eviction()
    refused("KAMERA_E_NULL", evict, e, scores=None)
    refused("KAMERA_E_ALIGN", evict, e, scores=FAKE + 2)
    refused("KAMERA_E_ALIGN", evict, e, kept=FAKE + 2)
    refused("KAMERA_E_SHAPE", evict, e, scores_stride=100 * 16 * 4 - 1)
    refused("KAMERA_E_SHAPE", evict, e, scores_stride=-1)
    need = step.evict_workspace_bytes(layout(), e)
    assert need > 0
    refused("KAMERA_E_WORKSPACE", evict, e, ws=(FAKE, need - 1))
    refused("KAMERA_E_WORKSPACE", evict, e, ws=None)
    refused("KAMERA_E_ALIGN", evict, e, ws=(FAKE + 64, need))
    refused("KAMERA_E_NULL", evict, e, pool=abi.make_pool(FAKE, None, 100))
    refused("KAMERA_E_SHAPE", evict, e, lay=layout(head_dim=7))
    refused("KAMERA_E_SHAPE", evict, eviction(heads_together=2), lay=layout(abi.MLA), pool=abi.make_pool(FAKE, None, 100))
    e.seqs["reserved"] = 1
    refused("KAMERA_E_SHAPE", evict, e)
    e = eviction()
    e.seqs["block_table"] = 0
    refused("KAMERA_E_NULL", evict, e)
    assert step.evict_workspace_bytes(layout(), eviction(keep=-1)) == 0
    with pytest.raises(ValueError):  # a table shorter than its tokens
        evict(eviction(tables=((1, 2),)))
    with pytest.raises(ValueError):
        eviction(keep=np.array([2 ** 32 + 20, 20]))
    evict(eviction(keep=40, first=90))  # all stay: nothing to do, whatever first and last are
    evict(eviction(tables=(), num_tokens=0, keep=0))
    with pytest.raises(abi.KameraError) as err:  # half a page each of one page: fine on the host (staging then needs a GPU)
        evict(eviction(tables=((1, 2, 3), (3, 4)), num_tokens=[40, 16], slot0=[0, 8], keep=10))
    assert err.value.name == "KAMERA_E_HIP"


def test_tensors_refused():
    import torch
    plan = plan_of(step.ATTEND | step.WEIGH | step.DIFFERENTIAL)
    bf, f32 = torch.bfloat16, torch.float32
    q, out, lse, scores = torch.zeros(1, 512, dtype=bf), torch.zeros(1, 512, dtype=bf), torch.zeros(1, 8), torch.zeros(100, 4, 16)
    for bad in (dict(q=q.float()), dict(q=torch.zeros(1, 511, dtype=bf)), dict(out=torch.zeros(1, 8, dtype=bf)), dict(lse=torch.zeros(1, 7)),
                dict(lambdas=torch.zeros(4, 63)), dict(lambdas=torch.zeros(4, 64, dtype=bf)), dict(norm_weight=torch.zeros(64, dtype=bf)),
                dict(norm_weight=torch.zeros(128, dtype=f32))):
        kw = dict(dict(q=q, out=out, lse=None, lambda_init=0.5), **bad)
        with pytest.raises(ValueError):
            step.attend_diff(plan, 0, kw.pop("q"), kw.pop("out"), 1.0, **kw)
    for bad in (dict(scores=torch.zeros(100, 4, 15)), dict(scores=scores.double()), dict(lse=lse.to(bf)), dict(scores=torch.zeros(100, 16, 4).transpose(1, 2))):
        kw = dict(dict(q=q, lse=lse, scores=scores), **bad)
        with pytest.raises(ValueError):
            step.weigh(plan, 0, kw["q"], kw["lse"], kw["scores"], 1.0)
    for kw in (dict(scores=torch.zeros(1, 100, 4, 16)), dict(scores=torch.zeros(2, 100, 4, 16, dtype=bf)),
               dict(scores=FAKE, kept=torch.zeros(2, 4, 39, dtype=torch.int32)), dict(scores=FAKE, kept=torch.zeros(2, 4, 40))):
        with pytest.raises(ValueError):
            evict(eviction(), **kw)


def test_scores_move_like_pages():
    for lay, heads in ((layout(), 4), (layout(abi.MLA), 1), (layout(num_kv_heads=3, head_dim=10, page_size=5), 3)):
        s = step.scores_layout(lay)
        assert s.family == abi.MLA and s.num_layers == 2 and s.page_size == lay.page_size
        assert (s.latent_dim + s.rope_dim) * 2 == 4 * heads  # bytes of a token's scores


# ------------------------------------------------------------------ the oracle against closed forms
def test_oracle_of_weights():
    """Against their own attention, a query's weights over the tokens it sees sum to one."""
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((5, 3, 8)), rng.standard_normal((20, 8))
    last = np.array([3, 19, -1, 0, 10])
    lse = so.attend(q, k, k, 0.3, last)[1]
    total, _ = eo.weights(q, k, lse, 0.3, last)
    assert np.isclose(total.sum(), 4 * 3) and (total[0] > 0) and np.allclose(eo.weights(q, k, lse, 0.3, np.minimum(last, 0))[0][1:], 0)
    one = eo.weights(q[3:4], k, lse[3:4], 0.3, last[3:4])[0]
    assert np.allclose(one[0], 3) and (one[1:] == 0).all()


def test_oracle_of_differential_heads():
    x = np.arange(6.0).reshape(2, 3)
    assert np.allclose(eo.combine(x, x, 1.0), 0) and np.allclose(eo.combine(x, 2 * x, 0.25), x / 2)
    v = np.zeros((4, 5))
    assert eo.lam(v, 0.3)[0] == 0.3 and eo.lam(None, 0.3)[0] == 0.3
    v[:2] = 1
    assert np.isclose(eo.lam(v, 0.0)[0], np.exp(5) - 1)
    y = eo.head_norm(x + 1, np.ones(3), 0.0, 1.0)
    assert np.allclose((y * y).mean(-1), 1) and (eo.head_norm(np.zeros((1, 3)), np.ones(3), 0.0, 1.0) == 0).all()


def test_oracle_of_evictions():
    s = np.array([5, 1, 1, 7, 1, 0, 2], np.float32)
    assert eo.stays(s, 4, 0, 0).tolist() == [0, 1, 3, 6] and eo.stays(s, 3, 1, 1).tolist() == [0, 3, 6] and eo.stays(s, 9, 9, 9).tolist() == list(range(7))
    assert eo.stays(s, 5, 0, 2).tolist() == [0, 1, 3, 5, 6] and eo.stays(s, 0, 0, 0).tolist() == []
    s[0] = np.nan
    s[1] = -np.inf
    assert eo.stays(s, 6, 0, 0).tolist() == [1, 2, 3, 4, 5, 6]
    big = np.array([[1e8, 1.0], [1.0, 1.0], [-1e8, 1.0]], np.float32)
    assert eo.group_scores(big).tolist() == [0.0, 3.0]  # in 32 bits, in the heads' order
    rows = np.random.default_rng(0).standard_normal((3, 6))
    y, _ = eo.turned(rows, np.array([0, 1, 5]), 1e4, 2)
    assert (y[:, :2] == rows[:, :2]).all() and np.allclose(y[0], rows[0])
    z = (rows[:, 2:4] + 1j * rows[:, 4:6]) * np.exp(-1j * np.array([0, 1, 5])[:, None] * 1e4 ** (-np.arange(2) / 2))
    assert np.allclose(y[:, 2:4] + 1j * y[:, 4:6], z)
